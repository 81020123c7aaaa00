"""Sums over very many tokens or rows: the longest chain of fp32 additions does not grow with them.  Terms that are all
alike round the same way at every step, the worst a chain can do.  2 to 45 GB on the device; skipped where that is not free."""
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F64 = torch.bfloat16, torch.float64


def _room(gb):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gb * 1e9:
        pytest.skip(f"needs {gb} GB of free device memory")


@pytest.mark.parametrize("T,d", [(3 << 26, 3), (1 << 24, 64), (1 << 22, 1001)])
def test_norm_weight_gradient_of_many_equal_rows(T, d):
    """A row's term is within 2^-22 of itself (three roundings); a chain has 4096 rows at most, then 16 row groups, 304
    blocks and the pieces of 4096 rows per group (at most 64 here): 2^-24 of the sum for each step."""
    _room(3 * 2 * T * d / 1e9 + 8)
    h = torch.ones((T, d), dtype=BF, device=DEV)
    dy = torch.full((T, d), 1 / 3, dtype=BF, device=DEV)
    gamma = torch.ones(d, device=DEV)
    rstd = torch.full((T,), 0.9, device=DEV)
    dgamma = mk.mk_moe_rmsnorm_bwd(dy, h, gamma, rstd)[1]
    want = T * float(dy[0, 0]) * float(rstd[0])
    assert bool(((dgamma.to(F64) / want - 1).abs() <= 2.0 ** -22 + (4096 + 16 + 304 + 64) * 2.0 ** -24).all()), \
        float((dgamma.to(F64) / want - 1).abs().max())


@pytest.mark.parametrize("T,d", [(3 << 26, 3), (1 << 22, 1001)])
def test_layer_norm_weight_gradients_of_many_equal_rows(T, d):
    """As above: dgamma's term is (x - mean) rstd dy, dbeta's dy."""
    _room(3 * 2 * T * d / 1e9 + 8)
    x = torch.ones((T, d), dtype=BF, device=DEV)
    dy = torch.full((T, d), 1 / 3, dtype=BF, device=DEV)
    gamma = torch.ones(d, device=DEV)
    mean, rstd = torch.full((T,), 0.25, device=DEV), torch.full((T,), 0.9, device=DEV)
    _, dgamma, dbeta = mk.mk_moe_layernorm_bwd(dy, x, gamma, mean, rstd)
    tol = 2.0 ** -22 + (4096 + 16 + 304 + 64) * 2.0 ** -24
    for got, term in ((dgamma, 0.75 * float(rstd[0]) * float(dy[0, 0])), (dbeta, float(dy[0, 0]))):
        assert bool(((got.to(F64) / (T * term) - 1).abs() <= tol).all()), float((got.to(F64) / (T * term) - 1).abs().max())


def test_norm_weight_gradient_in_pieces_is_the_rows_own():
    """More rows than one piece, values of both signs and a ragged end: every row counts once, dx is each row's own."""
    _room(12)
    T, d = (1 << 23) + 4099, 65
    g = torch.Generator(DEV).manual_seed(1)
    h = torch.empty((T, d), dtype=BF, device=DEV).normal_(generator=g)
    dy = torch.empty((T, d), dtype=BF, device=DEV).normal_(generator=g)
    gamma = 1 + 0.1 * torch.randn(d, generator=g, device=DEV)
    rstd = mk.mk_moe_rmsnorm(h, gamma)["rstd"]
    dx, dgamma = mk.mk_moe_rmsnorm_bwd(dy, h, gamma, rstd, dres=dy)
    want, mag = torch.zeros(d, dtype=F64, device=DEV), torch.zeros(d, dtype=F64, device=DEV)
    for a in range(0, T, 1 << 20):
        b = min(a + (1 << 20), T)
        t = dy[a:b].to(F64) * h[a:b].to(F64) * rstd[a:b].to(F64)[:, None]
        want += t.sum(0)
        mag += t.abs().sum(0)
        part = mk.mk_moe_rmsnorm_bwd(dy[a:b].clone(), h[a:b].clone(), gamma, rstd[a:b].clone(), dres=dy[a:b].clone())[0]
        assert torch.equal(part, dx[a:b]), a
    assert bool(((dgamma.to(F64) - want).abs() <= mag * (2.0 ** -22 + (4096 + 16 + 304 + 64) * 2.0 ** -24)).all())
    again = mk.mk_moe_rmsnorm_bwd(dy, h, gamma, rstd, dres=dy)[1]
    assert torch.equal(again, dgamma)


@pytest.mark.parametrize("T,E", [(3 << 28, 3), (3 << 28, 9), (1 << 24, 100)])
def test_router_losses_of_many_equal_tokens(T, E):
    """p = 1 / E and lse = log E for every token, each within 2^-21 of itself.  A lane adds 2048 tokens at most, then
    come 16 groups, 2048 partial rows a slice and 32 slices, and for the losses a tree: 2^-24 of the sum each."""
    _room(4 * T * E / 1e9 + 12)
    logits = torch.zeros((T, E), device=DEV)
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    loss, counts, probs = mk.mk_moe_balance_loss(logits, ids)
    assert counts[0].tolist() == [T] + [0] * (E - 1)
    tol = 2.0 ** -20 + (2048 + 16 + 2048 + 32 + 64) * 2.0 ** -24
    assert bool(((probs.to(F64) * E - 1).abs() <= tol).all()), float((probs.to(F64) * E - 1).abs().max())
    # sum_e E counts_e / T probs_e = E probs_0
    assert abs(float(loss[0]) - 1) <= tol + 2.0 ** -21
    lse2 = float(torch.log(torch.tensor(float(E), dtype=F64)) ** 2)
    assert abs(float(loss[1]) / lse2 - 1) <= tol + 2.0 ** -20
