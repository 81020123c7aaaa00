"""Codes in 8 bits are those of the fp32 quotient: each is the code nearest to value / scale, but for quotients that
lie within fp32's roundings of the middle between two codes."""
import pytest
import torch

import _ops8_ref as ref
import dispatch_ffn_combine_gb300 as mk

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3 = torch.float8_e4m3fn


def _quotients(v, scales, rows=1):
    """The codes of v [R, c] (fp32) over scales [ceil(R / rows), pitch], by a division in fp32 and torch's rounding."""
    R, c = v.shape
    s = scales.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :c]
    return (v / s).clamp(-448, 448).to(E4M3).view(torch.uint8)


def _scale(amax):
    """amax / 448 in fp32 (by a tensor: torch multiplies by a number's reciprocal)."""
    return (amax / torch.full_like(amax, 448.0)).clamp(min=2.0 ** -126)


def _same_codes(a, b):
    """Equal as values: 0 and -0 are."""
    return torch.equal(a.view(E4M3).float(), b.view(E4M3).float())


def _bf16_values(seed, blocks, low=-126, high=127):
    """Blocks of 128 bf16 values of all magnitudes up to 12 powers of two below a power between `low` and `high`."""
    g = torch.Generator(DEV).manual_seed(seed)
    top = torch.randint(low, high, (blocks, 1), generator=g, device=DEV)
    e = (top - torch.randint(0, 13, (blocks, 128), generator=g, device=DEV)).clamp(min=-126)
    m = 1 + torch.randint(0, 128, (blocks, 128), generator=g, device=DEV) / 128
    sign = 1 - 2 * torch.randint(0, 2, (blocks, 128), generator=g, device=DEV)
    return (sign * m.to(F64) * torch.exp2(e.to(F64))).to(BF)


def test_rows_are_the_fp32_quotients():
    """33 million values under scales of every magnitude, of which a quotient off by a unit moves some across a middle."""
    x = torch.cat([_bf16_values(s, 1 << 16) for s in range(4)]).view(-1, 512)
    codes, scales = mk.mk_moe_quant8_rows(x)
    assert torch.equal(scales, _scale(x.float().view(-1, 4, 128).abs().amax(2)))
    assert _same_codes(codes, _quotients(x.float(), scales))


@pytest.mark.parametrize("top", [-100, -110, -120, 100, 126])
def test_rows_of_very_small_and_large_values(top):
    x = _bf16_values(top + 200, 4096, top, top + 1).view(-1, 256)
    codes, scales = mk.mk_moe_quant8_rows(x)
    assert _same_codes(codes, _quotients(x.float(), scales[:, :2]))


def test_weights_are_the_fp32_quotients():
    E, n, d = 4, 256, 16384
    w = _bf16_values(9, E * n * d // 128, -20, 20).view(E, n, d)
    codes, scales = mk.mk_moe_quant8_weights(w)
    for e in range(E):
        amax = w[e].float().view(n // 128, 128, d // 128, 128).abs().amax((1, 3))
        assert torch.equal(scales[e], _scale(amax))
        assert _same_codes(codes[e], _quotients(w[e].float(), scales[e], 128))


def _nearest(codes, scales, v, slack):
    """Every code is the one nearest to v / scale for the exact v [R, c] (64 bits), or v / scale is within `slack` of
    itself to the middle of that code and its neighbour."""
    z = v / scales.to(F64).repeat_interleave(128, 1)[:, :v.shape[1]]
    _, e = torch.frexp(z)
    step = torch.exp2((e.to(F64) - 4).clamp(min=-9.0))
    got = ref.e4m3_values(codes.device)[codes.long()]
    off = (got - z).abs()
    # half a step of z's binade; a code at the binade's lower end is nearer to what lies below it, which the
    # smaller step there accounts for
    assert bool((off <= step / 2 + slack * z.abs() + (z.abs() > 448) * (z.abs() - 448)).all()), float((off - step / 2).max())
    return int((off > step / 2).sum())


# SwiGLU in fp32 for bf16 gates, in units of 2^-24 of the value: the exponential 4 (ex2's 2^-22), 1.5 for the two factors
# it is the product of (the second, 1 - g b, leaves out (g b)^2 / 2 < 2^-23.4) and 1 for their product's rounding; the sum
# with 1, the quotient and the product with up 1 each: 9.5.  The quotient by the scale is one more, and so is the scale.
SWIGLU = 10.51 * 2.0 ** -24


def _check_swiglu(gate, up, codes, scales):
    gate, up = gate.to(F64), up.to(F64)
    v = gate * torch.special.expit(gate) * up
    amax = v.unflatten(1, (-1, 128)).abs().amax(2)
    s = scales[:, :amax.shape[1]].to(F64)
    assert bool(((s - amax / 448).abs() <= SWIGLU * amax / 448).all())
    _nearest(codes, scales[:, :amax.shape[1]], v, SWIGLU)


@pytest.mark.parametrize("spread", [1.0, 6.0, 20.0])
def test_swiglu8_is_the_fp32_form(spread):
    S, f = 16384, 2048
    g = torch.Generator(DEV).manual_seed(3)
    gate = (torch.randn((S, f), generator=g, device=DEV) * spread).to(BF)
    up = torch.randn((S, f), generator=g, device=DEV).to(BF)
    codes, scales = mk.mk_moe_swiglu8(gate, up)
    for a in range(0, S, 4096):
        _check_swiglu(gate[a:a + 4096], up[a:a + 4096], codes[a:a + 4096], scales[a:a + 4096])


def test_swiglu8_of_every_gate():
    """All finite bf16 gates above -88.7 (below, exp(-g) is past fp32 and the form is zero), each beside ups that bring
    its product to one size, so that the codes of a block differ by the gates' errors."""
    bits = torch.arange(1 << 16, device=DEV, dtype=torch.int32)
    gate = bits.to(torch.int16).view(BF)
    gate = gate[torch.isfinite(gate) & (gate > -88.7) & (gate != 0)]
    silu = gate.to(F64) * torch.special.expit(gate.to(F64))
    gate, silu = gate[silu.abs() >= 2.0 ** -124], silu[silu.abs() >= 2.0 ** -124]
    for factor in (1.0, 1.3, 1.7):
        up = (factor / silu).to(F32).to(BF)
        ok = torch.isfinite(up) & (up.abs() >= 2.0 ** -126)
        n = int(ok.sum()) // 128 * 128
        a, b = gate[ok][:n].view(-1, 128), up[ok][:n].view(-1, 128)
        _check_swiglu(a, b, *mk.mk_moe_swiglu8(a, b))


def test_swiglu8_of_gates_whose_sigmoid_is_subnormal():
    """exp(-g) is finite down to g = -88.72, so the fp32 form has a value there; with ups of 2^120 it counts."""
    gate = torch.tensor([-80.0, -86.5, -87.0, -87.5, -88.0, -88.5] * 64, device=DEV).to(BF).view(3, 128)
    up = torch.full_like(gate, 2.0 ** 120)
    up[1] = 2.0 ** 126
    up[2, ::2] = -(2.0 ** 125)
    _check_swiglu(gate, up, *mk.mk_moe_swiglu8(gate, up))


@pytest.mark.parametrize("x_type", [BF, F32])
def test_norm_codes_are_the_fp32_quotients(x_type):
    """y = (h rstd) gamma in fp32 with the rstd that the call gives: two roundings, and one of the quotient."""
    T, d = 4096, 7168
    g = torch.Generator(DEV).manual_seed(5)
    x = (torch.randn((T, d), generator=g, device=DEV) * torch.exp(torch.randn(d, generator=g, device=DEV))).to(x_type)
    gamma = 1 + 0.3 * torch.randn(d, generator=g, device=DEV)
    r = mk.mk_moe_rmsnorm(x, gamma, bits8=True)
    for a in range(0, T, 1024):
        y = x[a:a + 1024].to(F64) * r["rstd"][a:a + 1024].to(F64)[:, None] * gamma.to(F64)
        _nearest(r["codes"][a:a + 1024], r["scales"][a:a + 1024], y, 3.01 * 2.0 ** -24)
        amax = y.view(1024, d // 128, 128).abs().amax(2)
        assert bool(((r["scales"][a:a + 1024].to(F64) - amax / 448).abs() <= 3.01 * 2.0 ** -24 * amax / 448).all())
