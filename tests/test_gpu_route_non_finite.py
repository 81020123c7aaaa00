"""GPU: NaN and infinite logits still give every token k valid, distinct
experts (NaN ranks last), leave the other tokens' routing bit for bit as it
was, and show in the weights.  Both routers, the one without a workspace and
the fused path's."""
import numpy as np
import pytest
import torch

import dispatch_ffn_combine_gb300 as mk
from dispatch_ffn_combine_gb300.workloads import CONFIGS, make_inputs

pytestmark = pytest.mark.gpu


def _inputs(T, d, E):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn((T, d), generator=g).to(torch.bfloat16).cuda()
    wg = (torch.randn((E, d), generator=g) * d ** -0.5).cuda()
    return x, wg


def _check_valid(ids, counts, E):
    i = np.sort(ids.cpu().numpy(), axis=1)
    assert i.min() >= 0 and i.max() < E
    assert (np.diff(i, axis=1) > 0).all()
    np.testing.assert_array_equal(counts.cpu().numpy(), np.bincount(i.ravel(), minlength=E))


# the last two take the tensor-core candidate filter (T >= 2048 and T d E >= 2^32)
@pytest.mark.parametrize("T,d,E,k", [(5, 64, 3, 3), (40, 128, 12, 3), (33, 256, 32, 4), (20, 128, 256, 8),
                                     (2048, 8192, 256, 8), (4096, 4096, 256, 1)])
def test_route_with_nan_tokens(T, d, E, k):
    x, wg = _inputs(T, d, E)
    ids0, w0, _ = mk.mk_moe_route(x, wg, None, k)
    broken = [0, T // 2, T - 1]
    bad = x.clone()
    bad[broken[0]] = float("nan")
    bad[broken[1], 3] = float("inf")
    bad[broken[2], 1] = float("nan")
    ids, w, counts = mk.mk_moe_route(bad, wg, None, k)
    _check_valid(ids, counts, E)
    keep = torch.ones(T, dtype=torch.bool, device=x.device)
    keep[broken] = False
    assert torch.equal(ids[keep], ids0[keep]) and torch.equal(w[keep], w0[keep])
    if k > 1:
        assert bool(torch.isnan(w[broken[0]]).all()) and bool(torch.isnan(w[broken[2]]).all())
    if T * E <= 1 << 21:
        n_ids, n_w = torch.empty_like(ids), torch.empty_like(w)
        n_counts = torch.empty_like(counts)
        mk.mk_moe_route_noalloc(bad, wg, None, k, n_ids, n_w, n_counts)
        _check_valid(n_ids, n_counts, E)
        assert torch.equal(n_ids, ids) and torch.equal(n_w.isnan(), w.isnan())


@pytest.mark.parametrize("T,d,E,k", [(50, 128, 32, 4), (2048, 8192, 256, 8)])
def test_route_with_a_nan_expert(T, d, E, k):
    """An expert whose gate row is NaN is chosen by no token; the others keep their order."""
    x, wg = _inputs(T, d, E)
    wg[E // 2] = float("nan")
    ids, w, counts = mk.mk_moe_route(x, wg, None, k)
    _check_valid(ids, counts, E)
    assert int(counts[E // 2]) == 0 and bool(torch.isfinite(w).all())
    without = wg.clone()
    without[E // 2] = 0.0
    bias = torch.zeros(E, device=x.device)
    bias[E // 2] = -1e30
    ids2, w2, _ = mk.mk_moe_route(x, without, bias, k)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


# the last takes the tensor-core candidate filter
@pytest.mark.parametrize("T,d,E,k,good", [(5, 64, 3, 3, 2), (40, 128, 12, 4, 1), (2048, 8192, 256, 8, 3)])
def test_route_shows_nan_logits_that_are_chosen(T, d, E, k, good):
    """Fewer numbers than k among a token's logits: NaN ones are chosen, and every weight of the token is NaN, as
    the softmax over them is.  Experts masked by -inf have the weight 0 and leave the others' as they are."""
    x, wg = _inputs(T, d, E)
    keep = torch.arange(0, E, E // good, device=x.device)[:good]
    drop = torch.ones(E, dtype=torch.bool, device=x.device)
    drop[keep] = False
    bad = wg.clone()
    bad[drop] = float("nan")
    ids, w, counts = mk.mk_moe_route(x, bad, None, k)
    _check_valid(ids, counts, E)
    assert bool(torch.isnan(w).all())
    assert torch.equal(ids[:, :good].sort(1).values, keep.to(torch.int32).expand(T, good))
    bias = torch.zeros(E, device=x.device)
    bias[drop] = float("-inf")
    ids, w, counts = mk.mk_moe_route(x, wg, bias, k)
    _check_valid(ids, counts, E)
    logits = x.double() @ wg[keep].double().t()
    want = torch.softmax(logits, 1).sort(1, descending=True).values
    # logits of size 5 at most, off by d 2^-23 of it, and a few fp32 operations
    torch.testing.assert_close(w[:, :good].double(), want, rtol=5 * d * 2.0 ** -23 + 1e-5, atol=1e-6)
    assert not bool(w[:, good:].any())
    if T * E <= 1 << 21:
        n_ids, n_w = torch.empty_like(ids), torch.empty_like(w)
        mk.mk_moe_route_noalloc(x, bad, None, k, n_ids, n_w)
        assert bool(torch.isnan(n_w).all())


@pytest.mark.parametrize("path", [mk.MK_PATH_STEPS, mk.MK_PATH_TILES, mk.MK_PATH_FUSED])
def test_layer_shows_nan_logits_that_are_chosen(path):
    """One gate row of numbers and k > 1: the NaN experts that each token also gets show in its output."""
    cfg = CONFIGS["ragged"]
    assert cfg.k > 1
    inp = make_inputs(cfg, seed=0, device="cuda")
    wg = inp["wg"].clone()
    wg[1:] = float("nan")
    ws = mk.alloc_workspace(cfg.T, cfg.d, cfg.E, cfg.k, cfg.f)
    y = mk.mk_moe_layer(inp["x"], wg, inp["bias"], inp["w1"], inp["w3"], inp["w2"], cfg.k, ws=ws, path=path)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    assert bool(torch.isnan(y).all())


@pytest.mark.parametrize("path", [mk.MK_PATH_STEPS, mk.MK_PATH_TILES, mk.MK_PATH_FUSED])
def test_layer_with_a_nan_token(path):
    cfg = CONFIGS["ragged"]
    inp = make_inputs(cfg, seed=0, device="cuda")
    x = inp["x"].clone()
    args = (inp["wg"], inp["bias"], inp["w1"], inp["w3"], inp["w2"], cfg.k)
    ws = mk.alloc_workspace(cfg.T, cfg.d, cfg.E, cfg.k, cfg.f)
    x[7] = float("nan")
    y = mk.mk_moe_layer(x, *args, ws=ws, path=path)
    assert mk.mk_moe_last_device_error(ws)[0] == mk.MK_OK
    clean = mk.mk_moe_layer(inp["x"], *args, ws=ws, path=path)
    keep = torch.arange(cfg.T, device=x.device) != 7
    assert bool(torch.isnan(y[7]).all()) and torch.equal(y[keep], clean[keep])
