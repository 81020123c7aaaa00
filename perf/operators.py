"""What is measured of the layer's training operators: their cases, inputs, plain forms and 64-bit definitions.

The operators are the pieces a training step needs beside the forward layer:

  dgrad    input gradient of the grouped expert GEMM (one weight, or the gate and up weights together)
  wgrad    weight gradient of the grouped expert GEMM (ragged rows per expert; fp32 or bf16, overwriting or accumulating)
  ckpt     tokens kept as 8-bit codes with a scale per 32 values, and restored straight into dispatched rows
  swiglu   SwiGLU that keeps gate and up in 8 bits, and its backward pass from that checkpoint
  norm     layer norm, forward and backward, with the gradients of its weight and bias

``own`` False computes them with elementary torch operations in 32 bits; True calls the framework's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest layer's backward: latency counts
        dict(name="dgrad tiny gate+up", op="dgrad", S=512, E=8, n=512, d=256, parts=2, zipf=0.0),
        # the mid layer's dx = dgate W1 + dup W3
        dict(name="dgrad mid gate+up", op="dgrad", S=16384, E=32, n=1408, d=2048, parts=2, zipf=0.0),
        # the skewed layer's down projection: experts from none or a few rows to tens of thousands
        dict(name="dgrad skewed down", op="dgrad", S=131072, E=64, n=4096, d=1536, parts=1, zipf=1.2),
        # the smallest layer's weight gradient
        dict(name="wgrad tiny", op="wgrad", S=512, E=8, n=512, d=256, out="fp32", accumulate=False, zipf=0.0),
        # the skewed layer's gate gradient added into the fp32 gradient of earlier micro-batches
        dict(name="wgrad skewed accumulate", op="wgrad", S=131072, E=64, n=1536, d=4096, out="fp32", accumulate=True,
             zipf=1.2),
        # many experts with about 32 rows each: bound by writing the gradient
        dict(name="wgrad many experts bf16", op="wgrad", S=8191, E=256, n=1408, d=2048, out="bf16", accumulate=False,
             zipf=0.0),
        # tokens of the smallest layer
        dict(name="ckpt tiny", op="ckpt", T=256, d=256, k=2),
        # tokens of the large layer, each restored into its eight dispatched rows
        dict(name="ckpt large", op="ckpt", T=32768, d=7168, k=8),
        # a ragged batch of a small layer
        dict(name="swiglu ragged", op="swiglu", S=3000, f=320),
        # all dispatched rows of the large layer
        dict(name="swiglu large", op="swiglu", S=262144, f=2048),
        # a ragged batch with a row length that no vector width divides, residual stream in fp32
        dict(name="norm ragged", op="norm", T=777, d=1001, x="fp32", residual=True),
        # the norm ahead of the large layer
        dict(name="norm large", op="norm", T=32768, d=7168, x="bf16", residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _m64(rng, lo, hi):
    return max(64, 64 * int(round(_log(rng, lo, hi) / 64)))


def draw(rng):
    op = rng.choice(["dgrad", "dgrad", "wgrad", "wgrad", "ckpt", "swiglu", "norm"])
    if op in ("dgrad", "wgrad"):
        while True:
            S, E = _log(rng, 1, 131072), _log(rng, 1, 256)
            n, d = _m64(rng, 64, 4096), _m64(rng, 64, 4096)
            if S * n * d <= 131072 * 1536 * 4096 and E * n * d <= 256 * 1408 * 2048 and S * max(n, d) < 1 << 31:
                break
        zipf = rng.choice([0.0, 0.6, 1.2])
        if op == "dgrad":
            parts = 1 if S * n * d > 131072 * 1536 * 2048 else rng.choice([1, 2])
            return dict(op=op, S=S, E=E, n=n, d=d, parts=parts, zipf=zipf)
        out = rng.choice(["fp32", "fp32", "bf16"])
        big = E * n * d > 64 * 1536 * 4096  # accumulating moves four times what writing bf16 does
        return dict(op=op, S=S, E=E, n=n, d=d, out="bf16" if big else out,
                    accumulate=not big and out == "fp32" and rng.random() < 0.5, zipf=zipf)
    if op == "ckpt":
        while True:
            T, d, k = _log(rng, 1, 32768), _m64(rng, 64, 7168), rng.randint(1, 8)
            if T * d * k <= 32768 * 7168 * 8:
                return dict(op=op, T=T, d=d, k=k)
    if op == "swiglu":
        while True:
            S, f = _log(rng, 1, 262144), _m64(rng, 64, 4096)
            if S * f <= 262144 * 2048:
                return dict(op=op, S=S, f=f)
    T, d = _log(rng, 1, 32768), _log(rng, 16, 7168)
    return dict(op=op, T=T, d=d, x=rng.choice(["bf16", "fp32"]) if T * d <= 16384 * 7168 else "bf16",
                residual=rng.random() < 0.5 and T * d <= 16384 * 7168)


def _counts(case, seed):
    """Rows of each expert: S draws over the experts, uniform or Zipf; ragged, and without rows for some."""
    g = torch.Generator().manual_seed(seed)
    p = 1.0 / torch.arange(1, case["E"] + 1, dtype=torch.float64) ** case["zipf"]
    p = p[torch.randperm(case["E"], generator=g)]
    picks = torch.multinomial(p, case["S"], replacement=True, generator=g)
    return torch.bincount(picks, minlength=case["E"])


def work(case):
    op = case["op"]
    if op in ("dgrad", "wgrad"):
        S, E, n, d = case["S"], case["E"], case["n"], case["d"]
        if op == "dgrad":
            touched = min(E, S)
            return {"bytes": case["parts"] * (2 * S * n + 2 * touched * n * d) + 2 * S * d,
                    "flops": 2 * case["parts"] * S * n * d}
        size = 4 if case["out"] == "fp32" else 2
        return {"bytes": 2 * S * (n + d) + E * n * d * size * (2 if case["accumulate"] else 1), "flops": 2 * S * n * d}
    if op == "ckpt":  # save: tokens in, codes and scales out; restore: codes and scales in, rows out
        one = case["T"] * case["d"]
        return {"bytes": 2 * one + 2 * (one + one // 32) + 2 * one * case["k"] + 4 * case["T"] * case["k"], "flops": 0}
    if op == "swiglu":
        one = case["S"] * case["f"]
        fwd = 4 * one + 2 * one + 2 * (one + one // 32)
        bwd = 2 * one + 2 * (one + one // 32) + 6 * one + 8 * case["S"]
        return {"bytes": fwd + bwd, "flops": 0}
    one, size = case["T"] * case["d"], 4 if case["x"] == "fp32" else 2
    return {"bytes": one * (size + 2) + one * (2 + 2 * size + (size if case["residual"] else 0)) + 16 * case["d"],
            "flops": 0}


# ------------------------------------------------------------------ inputs

def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _expert_weights(g, E, n, d):
    w = torch.empty((E, n, d), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 28) // (n * d))
    for e in range(0, E, step):
        w[e:e + step] = _normal(g, tuple(w[e:e + step].shape), d ** -0.5)
    return w


def _channels(g, d):
    """Spread of an activation's channels: log-normal, so that some stand out."""
    return torch.exp(0.7 * torch.randn(d, generator=g, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], dict(case)
    if op in ("dgrad", "wgrad"):
        S, E, n, d = case["S"], case["E"], case["n"], case["d"]
        counts = _counts(case, seed)
        s["counts"] = counts.tolist()
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).to(DEV)
        s["dout"] = _normal(g, (S, n), 0.05)
        if op == "dgrad":
            s["w"] = _expert_weights(g, E, n, d)
            s["dout2"] = _normal(g, (S, n), 0.05) if case["parts"] == 2 else None
            s["w2"] = _expert_weights(g, E, n, d) if case["parts"] == 2 else None
        else:
            s["x_perm"] = _normal(g, (S, d))
            s["dw"] = None
            if case["accumulate"]:
                s["dw"] = torch.randn((E, n, d), generator=g, device=DEV, dtype=torch.float32)
        return s
    if op == "ckpt":
        T, d, k = case["T"], case["d"], case["k"]
        s["x"] = (_normal(g, (T, d), dtype=torch.float32) * _channels(g, d)).to(torch.bfloat16)
        # each token's k rows among the dispatched ones: a permutation that keeps token order inside 64 groups
        group = torch.randint(0, 64, (T * k,), generator=g, device=DEV)
        slot = torch.empty(T * k, dtype=torch.int32, device=DEV)
        slot[torch.argsort(group, stable=True)] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        s["slot_row"] = slot.view(T, k)
        return s
    if op == "swiglu":
        S, f = case["S"], case["f"]
        c = _channels(g, f)
        s["gate"] = torch.empty((S, f), dtype=torch.bfloat16, device=DEV)
        s["up"], s["dh"] = torch.empty_like(s["gate"]), torch.empty_like(s["gate"])
        step = max(1, (1 << 28) // f)
        for r in range(0, S, step):
            m = min(step, S - r)
            s["gate"][r:r + m] = (_normal(g, (m, f), dtype=torch.float32) * c).to(torch.bfloat16)
            s["up"][r:r + m] = (_normal(g, (m, f), dtype=torch.float32) * c).to(torch.bfloat16)
            s["dh"][r:r + m] = _normal(g, (m, f), 0.01)
        s["row_weight"] = torch.rand(S, generator=g, device=DEV)
        return s
    T, d = case["T"], case["d"]
    dtype = torch.float32 if case["x"] == "fp32" else torch.bfloat16
    s["x"] = (_normal(g, (T, d), dtype=torch.float32) * _channels(g, d) + 0.1).to(dtype)
    s["gamma"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    s["beta"] = 0.1 * torch.randn(d, generator=g, device=DEV)
    s["dy"] = _normal(g, (T, d), 0.05)
    s["dres"] = _normal(g, (T, d), 0.05, dtype) if case["residual"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _plain_round8(v):
    """Blocks of 32 along the last axis through 8 bits and back: [..., c] fp32 -> [..., c] fp32."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    finite = torch.isfinite(b)
    amax = torch.where(finite, b.abs(), torch.zeros_like(b)).amax(-1, keepdim=True)
    m, e = torch.frexp(amax)
    q = torch.where(m > 0.875, e - 8, e - 9)
    q = torch.where(amax > 0, q, torch.full_like(q, -124)).clamp(min=-124)
    r = torch.ldexp(torch.ldexp(b, -q).to(torch.float8_e4m3fn).float(), q)
    return torch.where(finite, r, torch.full_like(r, math.nan)).reshape(v.shape)


def _plain(s):
    op = s["op"]
    if op == "dgrad":
        rows = zip(torch.split(s["dout"], s["counts"]), s["w"])
        dx = torch.cat([a.float() @ w.float() for a, w in rows])
        if s["dout2"] is not None:
            rows = zip(torch.split(s["dout2"], s["counts"]), s["w2"])
            dx += torch.cat([a.float() @ w.float() for a, w in rows])
        return {"dx": dx.to(torch.bfloat16)}
    if op == "wgrad":
        rows = zip(torch.split(s["dout"], s["counts"]), torch.split(s["x_perm"], s["counts"]))
        dw = torch.stack([a.float().t() @ x.float() for a, x in rows])
        if s["accumulate"]:
            s["dw"] += dw
            return {"dw": s["dw"]}
        return {"dw": dw if s["out"] == "fp32" else dw.to(torch.bfloat16)}
    if op == "ckpt":
        x8 = _plain_round8(s["x"].float()).to(torch.bfloat16)
        x_perm = torch.empty((s["T"] * s["k"], s["d"]), dtype=torch.bfloat16, device=x8.device)
        x_perm[s["slot_row"].reshape(-1).long()] = x8.repeat_interleave(s["k"], 0)
        return {"x_perm": x_perm}
    if op == "swiglu":
        g, u, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
        h = g / (1 + torch.exp(-g)) * u
        g, u = _plain_round8(g), _plain_round8(u)
        sig = 1 / (1 + torch.exp(-g))
        a = g * sig
        w = s["row_weight"][:, None]
        return {"h": h.to(torch.bfloat16), "dgate": (w * dh * u * sig * (1 + g * (1 - sig))).to(torch.bfloat16),
                "dup": (w * dh * a).to(torch.bfloat16), "hw": (w * a * u).to(torch.bfloat16),
                "drow_weight": (dh * a * u).sum(1)}
    x, dy = s["x"].float(), s["dy"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    xh = c * rstd[:, None]
    y = xh * s["gamma"] + s["beta"]
    t = dy * s["gamma"]
    dx = rstd[:, None] * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"y": y.to(torch.bfloat16), "mean": mean, "rstd": rstd, "dx": dx.to(s["x"].dtype),
            "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def run(state):
    if not own:
        return _plain(state)
    import dispatch_ffn_combine_gb300 as mk

    s, op = state, state["op"]
    if op == "dgrad":
        return {"dx": mk.mk_moe_grouped_dgrad(s["dout"], s["offsets"], s["w"], dout2=s["dout2"], w2=s["w2"])}
    if op == "wgrad":
        dtype = torch.float32 if s["out"] == "fp32" else torch.bfloat16
        return {"dw": mk.mk_moe_grouped_wgrad(s["dout"], s["offsets"], s["x_perm"], dw=s["dw"],
                                              accumulate=s["accumulate"], dtype=dtype)}
    if op == "ckpt":
        codes, scales = mk.mk_moe_ckpt8_save(s["x"])
        return {"x_perm": mk.mk_moe_ckpt8_dispatch(codes, scales, s["slot_row"])}
    if op == "swiglu":
        h, codes, scales = mk.mk_moe_swiglu_ckpt8(s["gate"], s["up"])
        dgate, dup, hw, drw = mk.mk_moe_swiglu_ckpt8_bwd(s["dh"], codes, scales, s["row_weight"])
        return {"h": h, "dgate": dgate, "dup": dup, "hw": hw, "drow_weight": drw}
    y, mean, rstd = mk.mk_moe_layernorm(s["x"], s["gamma"], s["beta"], EPS)
    dx, dgamma, dbeta = mk.mk_moe_layernorm_bwd(s["dy"], s["x"], s["gamma"], mean, rstd, dres=s["dres"])
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}


# ------------------------------------------------------------------ definitions in 64 bits

def _nearest8(v):
    """bf16 tensor [R, c] -> the fp64 values its 8-bit form stands for, from the format's definition: a block of 32
    shares the smallest power of two (2^-124 at least) that brings its largest finite magnitude to 448 or below; a
    value becomes the nearest multiple of 2^(e - 3) for e its binary exponent, 2^-9 at least, ties to even."""
    R, c = v.shape
    b = v.double().view(R, c // 32, 32)
    big = torch.where(b.abs() < math.inf, b.abs(), torch.zeros_like(b)).max(dim=2, keepdim=True).values
    q = torch.ceil(torch.log2(torch.clamp(big, min=2.0 ** -140) / 448.0))
    q = torch.where(big > 448.0 * torch.exp2(q), q + 1, q)
    q = torch.where(big <= 448.0 * torch.exp2(q - 1), q - 1, q)
    scale = torch.exp2(torch.clamp(q, min=-124.0))
    z = b / scale
    e = torch.floor(torch.log2(torch.clamp(z.abs(), min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > z.abs().clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= z.abs(), e + 1, e)
    step = torch.exp2(torch.clamp(e - 3, min=-9.0))
    return (torch.round(z / step) * step * scale).view(R, c)


def _by_rows(f, rows, step):
    """The pieces of f(r0, r1) over row ranges, joined output by output."""
    parts = [f(r, min(r + step, rows)) for r in range(0, rows, step)]
    return [torch.cat(p) for p in zip(*parts)]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("dgrad", "wgrad"):
        if work(case)["flops"] > 6e12:  # 64-bit products run at about 1 TFLOP/s
            return None
        S, E, n, d = case["S"], case["E"], case["n"], case["d"]
        r = 0
        if op == "dgrad":
            dx = torch.zeros((S, d), dtype=torch.float64, device=DEV)
            for e, c in enumerate(s["counts"]):
                if c:
                    torch.mm(s["dout"][r:r + c].double(), s["w"][e].double(), out=dx[r:r + c])
                    if s["dout2"] is not None:
                        dx[r:r + c].addmm_(s["dout2"][r:r + c].double(), s["w2"][e].double())
                r += c
            return {"dx": dx}
        dw = s["dw"].double() if case["accumulate"] else torch.zeros((E, n, d), dtype=torch.float64, device=DEV)
        for e, c in enumerate(s["counts"]):
            if c:
                dw[e].addmm_(s["dout"][r:r + c].double().t(), s["x_perm"][r:r + c].double())
            r += c
        return {"dw": dw}
    if op == "ckpt":
        T, k, d = case["T"], case["k"], case["d"]
        out = torch.empty((T * k, d), dtype=torch.float64, device=DEV)
        step = max(1, (1 << 26) // d)
        for t in range(0, T, step):
            v = _nearest8(s["x"][t:t + step])
            for j in range(k):
                out[s["slot_row"][t:t + step, j].long()] = v
        return {"x_perm": out}
    if op == "swiglu":
        def rows(a, b):
            g, u, dh = s["gate"][a:b].double(), s["up"][a:b].double(), s["dh"][a:b].double()
            w = s["row_weight"][a:b].double()[:, None]
            h = g * torch.special.expit(g) * u
            g, u = _nearest8(s["gate"][a:b]), _nearest8(s["up"][a:b])
            p = torch.special.expit(g)
            slope = p + g * p * (1 - p)
            return h, dh * w * u * slope, dh * w * g * p, w * g * p * u, torch.einsum("rf,rf->r", dh, g * p * u)
        h, dgate, dup, hw, drw = _by_rows(rows, case["S"], max(1, (1 << 25) // case["f"]))
        return {"h": h, "dgate": dgate, "dup": dup, "hw": hw, "drow_weight": drw}
    d = case["d"]
    gamma, beta = s["gamma"].double(), s["beta"].double()
    dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(beta)

    def rows(a, b):
        x, dy = s["x"][a:b].double(), s["dy"][a:b].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        inv = 1.0 / torch.sqrt(var + EPS)
        z = (x - mean) * inv
        dgamma.add_(torch.einsum("td,td->d", dy, z))
        dbeta.add_(dy.sum(0))
        dz = dy * gamma
        along = torch.einsum("td,td->t", dz, z)[:, None] / d
        dx = inv * (dz - dz.sum(1, keepdim=True) / d - along * z)
        if s["dres"] is not None:
            dx = dx + s["dres"][a:b].double()
        return z * gamma + beta, mean[:, 0], inv[:, 0], dx
    y, mean, rstd, dx = _by_rows(rows, case["T"], max(1, (1 << 25) // d))
    return {"y": y, "mean": mean, "rstd": rstd, "dx": dx, "dgamma": dgamma, "dbeta": dbeta}
