"""The training operators without a GPU: their 64-bit formulas against central
differences, and the entry points' refusals (before any CUDA call)."""
import ctypes

import pytest
import torch

import _training_ref as ref
import dispatch_ffn_combine_gb300 as mk
from dispatch_ffn_combine_gb300 import build as cuda_build

F64 = torch.float64


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return mk.load_library()


def _differences(f, x, h=1e-5):
    """Gradient of the scalar f at x by central differences."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        d = torch.zeros_like(x).view(-1)
        d[i] = h
        d = d.view(x.shape)
        g.view(-1)[i] = (f(x + d) - f(x - d)) / (2 * h)
    return g


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


# Central differences of step 1e-5 on functions with third derivatives of order 1 to 100: error
# about 1e-10 * 100 from the step and 1e-16 / 1e-5 from rounding; 1e-6 leaves two orders of room.
FD = dict(rtol=1e-6, atol=1e-6)


def test_grouped_gradients_match_differences():
    off = [0, 3, 3, 4, 8]
    x, w, c = _rand(8, 5, seed=1), _rand(4, 6, 5, seed=2), _rand(8, 6, seed=3)

    def loss(x, w):
        return sum((c[a:b] * (x[a:b] @ w[e].t())).sum() for e, (a, b) in enumerate(ref.spans(off)))

    torch.testing.assert_close(ref.dgrad(c, off, w), _differences(lambda v: loss(v, w), x), **FD)
    torch.testing.assert_close(ref.wgrad(c, off, x, 4), _differences(lambda v: loss(x, v), w), **FD)


def test_swiglu_gradients_match_differences():
    g, u, c, w = _rand(3, 4, seed=1) * 2, _rand(3, 4, seed=2), _rand(3, 4, seed=3), _rand(3, seed=4).abs()

    def loss(g, u, w):  # the row's weight multiplies what the activation feeds
        return (w[:, None] * c * ref.swiglu(g, u)).sum()

    dg, du, hw, dw = ref.swiglu_bwd(c, g, u, w)
    torch.testing.assert_close(dg, _differences(lambda v: loss(v, u, w), g), **FD)
    torch.testing.assert_close(du, _differences(lambda v: loss(g, v, w), u), **FD)
    torch.testing.assert_close(dw, _differences(lambda v: loss(g, u, v), w), **FD)
    torch.testing.assert_close(hw, w[:, None] * ref.swiglu(g, u))


def test_layernorm_gradients_match_differences():
    x, gamma, beta, c = _rand(3, 7, seed=1), _rand(7, seed=2), _rand(7, seed=3), _rand(3, 7, seed=4)

    def loss(x, gamma, beta):
        return (c * ref.layernorm(x, gamma, beta, 1e-3)[0]).sum()

    dx, dgamma, dbeta = ref.layernorm_bwd(c, x, gamma, 1e-3)
    torch.testing.assert_close(dx, _differences(lambda v: loss(v, gamma, beta), x), **FD)
    torch.testing.assert_close(dgamma, _differences(lambda v: loss(x, v, beta), gamma), **FD)
    torch.testing.assert_close(dbeta, _differences(lambda v: loss(x, gamma, v), beta), **FD)


def test_eight_bit_format_matches_torch_e4m3():
    """The searched format against torch's e4m3 rounding under the searched scale."""
    g = torch.Generator().manual_seed(5)
    x = (torch.randn((64, 96), generator=g) * torch.exp(3 * torch.randn((64, 96), generator=g))).to(torch.bfloat16)
    x[3, :32] = 0
    x[4, 5] = 448.0 * 64
    v, q = ref.round8(x)
    scale = torch.pow(2.0, q.to(F64)).repeat_interleave(32, 1)
    want = (x.to(F64) / scale).to(torch.float32).to(torch.float8_e4m3fn).to(F64) * scale
    assert torch.equal(v, want)
    assert bool((q[3, 0] == -124))


def _vp(v):
    return ctypes.c_void_p(v)


A = _vp(0x10000)  # never dereferenced: every case fails validation first
ODD = _vp(0x10008)  # not 16-byte aligned

# entry point -> (names, valid arguments); each refusal changes some of them
CALLS = {
    "mk_moe_grouped_dgrad": ("dout off w dout2 w2 S d E n dx ws wsb s".split(),
                             [A, A, A, A, A, 64, 128, 8, 192, A, A, 4096, None]),
    "mk_moe_grouped_wgrad": ("dout off x S d E n dw type acc ws wsb s".split(),
                             [A, A, A, 64, 128, 8, 192, A, 1, 0, A, 4096, None]),
    "mk_moe_ckpt8_save": ("x T d codes scales s".split(), [A, 64, 128, A, A, None]),
    "mk_moe_ckpt8_dispatch": ("codes scales slot T d k x ws wsb s".split(),
                              [A, A, A, 64, 128, 2, A, A, 4096, None]),
    "mk_moe_swiglu_ckpt8": ("gate up S f h codes scales s".split(), [A, A, 64, 128, A, A, A, None]),
    "mk_moe_swiglu_ckpt8_bwd": ("dh codes scales w S f dgate dup hw dw s".split(),
                                [A, A, A, A, 64, 128, A, A, A, A, None]),
    "mk_moe_layernorm": ("x type gamma beta T d eps y mean rstd s".split(),
                         [A, 0, A, A, 64, 100, 1e-5, A, A, A, None]),
    "mk_moe_layernorm_bwd": ("dy x type gamma mean rstd dres T d dx dgamma dbeta ws wsb s".split(),
                             [A, A, 0, A, A, A, A, 64, 100, A, A, A, A, 1 << 20, None]),
}
INVALID = {
    "mk_moe_grouped_dgrad": [dict(dout=None), dict(off=None), dict(w=None), dict(dx=None), dict(dout2=None),
                             dict(w2=None), dict(d=100), dict(n=96), dict(E=0), dict(E=257), dict(S=-1),
                             dict(dout=ODD), dict(w2=ODD), dict(dx=ODD)],
    "mk_moe_grouped_wgrad": [dict(dout=None), dict(off=None), dict(x=None), dict(dw=None), dict(d=100), dict(n=0),
                             dict(E=257), dict(S=-1), dict(type=2), dict(type=0, acc=1), dict(x=ODD), dict(dw=ODD),
                             dict(S=0, dw=None)],
    "mk_moe_ckpt8_save": [dict(x=None), dict(codes=None), dict(scales=None), dict(d=96), dict(T=-1), dict(x=ODD),
                          dict(codes=ODD)],
    "mk_moe_ckpt8_dispatch": [dict(codes=None), dict(scales=None), dict(slot=None), dict(x=None), dict(d=32),
                              dict(k=0), dict(k=9), dict(T=-1), dict(x=ODD)],
    "mk_moe_swiglu_ckpt8": [dict(gate=None), dict(up=None), dict(h=None), dict(codes=None), dict(scales=None),
                            dict(f=96), dict(S=-1), dict(up=ODD), dict(h=ODD)],
    "mk_moe_swiglu_ckpt8_bwd": [dict(dh=None), dict(codes=None), dict(scales=None), dict(dgate=None), dict(dup=None),
                                dict(f=0), dict(S=-1), dict(dh=ODD), dict(hw=ODD)],
    "mk_moe_layernorm": [dict(x=None), dict(gamma=None), dict(beta=None), dict(y=None), dict(mean=None),
                         dict(rstd=None), dict(type=3), dict(d=0), dict(T=-1), dict(eps=-1.0),
                         dict(eps=float("nan")), dict(x=ODD), dict(gamma=ODD)],
    "mk_moe_layernorm_bwd": [dict(dy=None), dict(x=None), dict(gamma=None), dict(mean=None), dict(rstd=None),
                             dict(dx=None), dict(dgamma=None), dict(dbeta=None), dict(type=-1), dict(d=0),
                             dict(dy=ODD), dict(dres=ODD), dict(T=0, dgamma=None)],
}
UNSUPPORTED = {
    "mk_moe_grouped_dgrad": [dict(S=1 << 31), dict(S=1 << 25, d=128)],
    "mk_moe_grouped_wgrad": [dict(S=1 << 31)],
    "mk_moe_ckpt8_save": [dict(T=1 << 31), dict(T=1 << 30, d=1024)],
    "mk_moe_ckpt8_dispatch": [dict(T=1 << 30, k=2), dict(T=1 << 28, d=1024, k=4)],
    "mk_moe_swiglu_ckpt8": [dict(S=1 << 31), dict(S=1 << 30, f=1024)],
    "mk_moe_swiglu_ckpt8_bwd": [dict(S=1 << 31)],
    "mk_moe_layernorm": [dict(d=16385), dict(T=1 << 31)],
    "mk_moe_layernorm_bwd": [dict(d=16385), dict(T=1 << 31)],
}
WORKSPACE = {
    "mk_moe_grouped_dgrad": [dict(ws=None), dict(ws=_vp(0x10080)), dict(wsb=256 + 4 * 9 - 1)],
    "mk_moe_grouped_wgrad": [dict(ws=None), dict(ws=_vp(0x10080)), dict(wsb=255)],
    "mk_moe_ckpt8_dispatch": [dict(ws=None), dict(wsb=255)],
    "mk_moe_layernorm_bwd": [dict(ws=None), dict(ws=_vp(0x10080)), dict(wsb=256)],
}
NO_ROWS = {  # valid calls that enqueue nothing
    "mk_moe_grouped_dgrad": dict(S=0), "mk_moe_ckpt8_save": dict(T=0), "mk_moe_ckpt8_dispatch": dict(T=0),
    "mk_moe_swiglu_ckpt8": dict(S=0), "mk_moe_swiglu_ckpt8_bwd": dict(S=0), "mk_moe_layernorm": dict(T=0),
}


def _call(lib, name, over):
    names, args = CALLS[name]
    args = list(args)
    for key, v in over.items():
        args[names.index(key)] = v
    return getattr(lib, name)(*args)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_training_entry_points_reject_bad_arguments(lib, name):
    for over in INVALID[name]:
        assert _call(lib, name, over) == mk.MK_ERR_INVALID_ARG, over
    for over in UNSUPPORTED[name]:
        assert _call(lib, name, over) == mk.MK_ERR_UNSUPPORTED, over
    for over in WORKSPACE.get(name, []):
        assert _call(lib, name, over) == mk.MK_ERR_WORKSPACE, over
    if name in NO_ROWS:
        assert _call(lib, name, NO_ROWS[name]) == mk.MK_OK


def test_layernorm_workspace_size(lib):
    assert mk.load_library().mk_moe_layernorm_bwd_workspace_size(32768, 7168) >= 2 * 7168 * 4
    assert lib.mk_moe_layernorm_bwd_workspace_size(0, 64) >= 256
    for bad in [(-1, 64), (4, 0), (4, 16385), (1 << 31, 64)]:
        assert lib.mk_moe_layernorm_bwd_workspace_size(*bad) == 0, bad


def test_binding_refuses_wrong_tensors():
    """The Python entry points name the tensor that is wrong (checked before the library is called)."""
    b = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must be"):
        mk.mk_moe_ckpt8_save(b.float())
    with pytest.raises(ValueError, match="x must be a CUDA"):
        mk.mk_moe_ckpt8_save(b)
    with pytest.raises(ValueError, match="x must have 2 dimensions"):
        mk.mk_moe_layernorm(b[0], torch.ones(64), torch.ones(64))
    with pytest.raises(TypeError, match="x must be torch.bfloat16 or torch.float32"):
        mk.mk_moe_layernorm(b.double(), torch.ones(64), torch.ones(64))
    with pytest.raises(ValueError, match="gate must be contiguous"):
        mk.mk_moe_swiglu_ckpt8(torch.zeros((4, 128), dtype=torch.bfloat16)[:, :64], b)
