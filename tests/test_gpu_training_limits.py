"""GPU: the training operators next to their size limits, where a 32-bit index
would wrap.  Some 40 to 70 GB on the device; skipped where that much is not free."""
import pytest
import torch

import _training_ref as ref
import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F64 = torch.float64
BF = torch.bfloat16
GUARD = 1 << 16  # values kept on either side of an output


def _room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip(f"needs {gb} GB of free device memory")


def _guarded(shape, dtype):
    """A tensor of NaNs inside a buffer of NaNs."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 2 * GUARD,), float("nan"), dtype=dtype, device=DEV)
    return buf, buf[GUARD:GUARD + n].view(shape)


def _untouched(buf):
    return bool(torch.isnan(buf[:GUARD]).all()) and bool(torch.isnan(buf[-GUARD:]).all())


def test_layernorm_with_the_most_rows():
    """2^31 - 1 rows: every row is normalised, and nothing outside the tensors is written (the walk over the
    rows looks past the last one).

    Tolerances: three values of size |x| summed in fp32, each step off by 2^-23 of the sum at most (1e-6 of the
    largest, as in the sums of longer rows); a few fp32 operations after that (1e-5 of the terms), then one
    rounding to bf16 (2^-8).  dy is zero but for the first 5000 and the last 20000 rows, so that the columns'
    sums have 25000 terms."""
    _room(110)
    T, d, eps = (1 << 31) - 1, 3, 1e-5
    x = torch.empty((T, d), dtype=BF, device=DEV)
    x.view(-1).normal_(0.5, 2.0, generator=torch.Generator(DEV).manual_seed(1))
    gamma = torch.tensor([0.75, 1.0, 1.5], device=DEV)
    beta = torch.tensor([0.25, -0.5, 0.0], device=DEV)
    (ybuf, y), (mbuf, mean), (rbuf, rstd) = (_guarded(s, t) for s, t in (((T, d), BF), ((T,), torch.float32),
                                                                          ((T,), torch.float32)))
    mk.mk_moe_layernorm(x, gamma, beta, eps, y=y, mean=mean, rstd=rstd)
    assert _untouched(ybuf) and _untouched(mbuf) and _untouched(rbuf)
    for a in range(0, T, 1 << 26):
        b = min(a + (1 << 26), T)
        wy, wm, wr = ref.layernorm(x[a:b], gamma, beta, eps)
        size = x[a:b].to(F64).abs().amax(1)
        assert bool(((mean[a:b] - wm).abs() <= 1e-6 * size + 2.0 ** -23 * wm.abs()).all()), a
        assert bool(((rstd[a:b] - wr).abs() <= 1e-5 * wr + 2.0 ** -23 * wr).all()), a
        slack = 1e-6 * (size * wr)[:, None] * gamma.abs() + 1e-5 * (wy.abs() + beta.abs())
        assert bool(((y[a:b] - wy).abs() <= 2.0 ** -8 * wy.abs() + slack).all()), a
    del ybuf, y
    dy = torch.zeros((T, d), dtype=BF, device=DEV)
    ends = [(0, 5000), (T - 20000, T)]
    for i, (a, b) in enumerate(ends):
        dy[a:b] = torch.randn((b - a, d), generator=torch.Generator().manual_seed(7 + i)).to(BF).to(DEV)
    dxbuf, dx = _guarded((T, d), BF)
    _, dgamma, dbeta = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd, dx=dx)
    assert _untouched(dxbuf)
    for a in range(5000, T - 20000, 1 << 28):
        assert not bool(dx[a:min(a + (1 << 28), T - 20000)].any()), a
    wg, wb, sg, sb = (torch.zeros(d, dtype=F64, device=DEV) for _ in range(4))
    for a, b in ends:
        wx, g, bt = ref.layernorm_bwd(dy[a:b], x[a:b], gamma, eps)
        _, wm, wr = ref.layernorm(x[a:b], gamma, beta, eps)
        xh = (x[a:b].to(F64) - wm[:, None]) * wr[:, None]
        size = x[a:b].to(F64).abs().amax(1, keepdim=True)
        err = 1e-6 * size * wr[:, None] + 1e-5 * xh.abs()  # of the normalised value
        t = dy[a:b].to(F64) * gamma.to(F64)
        along = (t * xh).abs().mean(1, keepdim=True)
        slack = wr[:, None] * (1e-5 * (t.abs() + t.abs().mean(1, keepdim=True) + xh.abs() * along)
                               + err * along + xh.abs() * (t.abs() * err).mean(1, keepdim=True))
        assert bool(((dx[a:b] - wx).abs() <= 2.0 ** -8 * wx.abs() + slack).all())
        wg, wb = wg + g, wb + bt
        sg = sg + (dy[a:b].to(F64).abs() * err).sum(0) + 25000 * 2.0 ** -23 * (dy[a:b].to(F64) * xh).abs().sum(0)
        sb = sb + 25000 * 2.0 ** -23 * dy[a:b].to(F64).abs().sum(0)
    assert bool(((dgamma - wg).abs() <= sg).all()) and bool(((dbeta - wb).abs() <= sb).all())


def test_swiglu_with_the_longest_row():
    """One row of 2^31 - 64 values: each is computed on its own, so a row that repeats a short one gives the
    short one's outputs over and over, bit for bit, and nothing outside the outputs is written."""
    _room(60)
    f = (1 << 31) - 64
    short = 64 * 31 * 601
    times = f // short
    assert times * short == f
    gate, up, dh = ((2 * torch.randn((1, short), generator=torch.Generator().manual_seed(i))).to(BF).to(DEV)
                    for i in range(3))
    w = torch.tensor([0.75], device=DEV)
    h, codes, scales = mk.mk_moe_swiglu_ckpt8(gate, up)
    want = mk.mk_moe_swiglu_ckpt8_bwd(dh, codes, scales, w)
    long_gate, long_up = gate.repeat(1, times), up.repeat(1, times)
    long_h, long_codes, long_scales = mk.mk_moe_swiglu_ckpt8(long_gate, long_up)
    assert bool((long_h.view(times, short) == h).all())
    for got, one in ((long_codes, codes), (long_scales, scales)):
        for plane in range(2):
            assert bool((got[plane].view(times, -1) == one[plane]).all())
    del long_gate, long_up, long_h
    outs = [_guarded((1, f), BF) for _ in range(3)]
    drow = mk.mk_moe_swiglu_ckpt8_bwd(dh.repeat(1, times), long_codes, long_scales, w, dgate=outs[0][1],
                                      dup=outs[1][1], hw=outs[2][1])[3]
    for (buf, t), one in zip(outs, want):
        assert _untouched(buf)
        assert bool((t.view(times, short) == one).all())
    assert bool(torch.isfinite(drow).all())
