"""GPU: the layer norm where a row group takes several rows one after the other:
lengths that are no multiple of 8, several groups per block, one ring stage."""
import pytest
import torch

import _training_ref as ref
import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F64 = torch.float64
BF = torch.bfloat16


def _within(got, want, unit, slack, what):
    over = (got.to(F64) - want).abs() - unit * want.abs() - slack
    assert float(over.max()) <= 0, f"{what}: over the bound by {float(over.max()):.3e}"


@pytest.mark.parametrize("T,d,dtype,residual",
                         [(20000, d, dt, res) for d in (3, 31, 1001, 4095) for dt, res in ((BF, False), (BF, True),
                                                                                           (torch.float32, True))] +
                         [(1000, 12289, torch.float32, True), (1000, 16384, torch.float32, True),
                          (3001, 4608, BF, False), (3001, 16376, BF, True)])
def test_layernorm_several_rows_per_group(T, d, dtype, residual):
    """Against 64 bits.  dy are whole numbers, so dbeta is exact and shows a row that is lost or taken twice.

    Tolerances: d values of size |x| summed in fp32 over threads and a tree (1e-6 of the largest), a few fp32
    operations (1e-5 of the terms), one rounding of what is stored (2^-8 bf16, 2^-23 fp32).  dgamma's chains of
    additions are a group's rows, its block's groups and the blocks: under 256, each off by 2^-24 of the terms."""
    g = torch.Generator().manual_seed(T + d)
    x = (2 * torch.randn((T, d), generator=g) + 0.5).to(dtype).to(DEV)
    dy = torch.randint(-3, 4, (T, d), generator=g).to(BF).to(DEV)
    dres = torch.randn((T, d), generator=g).to(dtype).to(DEV) if residual else None
    gamma = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    beta = (0.2 * torch.randn(d, generator=g)).to(DEV)
    eps = 1e-5
    unit = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    y, mean, rstd = mk.mk_moe_layernorm(x, gamma, beta, eps)
    dx, dgamma, dbeta = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd, dres=dres)
    assert torch.equal(dbeta.to(F64), dy.to(F64).sum(0))
    wg, sg = torch.zeros(d, dtype=F64, device=DEV), torch.zeros(d, dtype=F64, device=DEV)
    for a in range(0, T, 4000):
        b = min(a + 4000, T)
        wy, wm, wr = ref.layernorm(x[a:b], gamma, beta, eps)
        size = x[a:b].to(F64).abs().amax(1, keepdim=True)
        _within(mean[a:b], wm, 2.0 ** -23, 1e-6 * size[:, 0], "mean")
        _within(rstd[a:b], wr, 2.0 ** -23, 1e-5 * wr, "rstd")
        _within(y[a:b], wy, 2.0 ** -8, 1e-6 * size * wr[:, None] * gamma.abs() + 1e-5 * (wy.abs() + beta.abs()), "y")
        wx, dg, _ = ref.layernorm_bwd(dy[a:b], x[a:b], gamma, eps, dres[a:b] if residual else None)
        xh = (x[a:b].to(F64) - wm[:, None]) * wr[:, None]
        err = 1e-6 * size * wr[:, None] + 1e-5 * xh.abs()  # of the normalised value
        t = dy[a:b].to(F64) * gamma.to(F64)
        along = (t * xh).abs().mean(1, keepdim=True)
        slack = wr[:, None] * (1e-5 * (t.abs() + t.abs().mean(1, keepdim=True) + xh.abs() * along)
                               + err * along + xh.abs() * (t.abs() * err).mean(1, keepdim=True))
        if residual:
            slack = slack + 2.0 ** -23 * dres[a:b].to(F64).abs()
        _within(dx[a:b], wx, unit, slack, "dx")
        wg += dg
        sg += (dy[a:b].to(F64).abs() * err).sum(0) + 256 * 2.0 ** -24 * (dy[a:b].to(F64) * xh).abs().sum(0)
    _within(dgamma, wg, 2.0 ** -23, sg, "dgamma")
    again = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd, dres=dres)
    for p, q in zip((dx, dgamma, dbeta), again):
        assert torch.equal(p, q)
