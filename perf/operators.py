"""Cases of the RMSNorm (with the residual's addition and an MXFP8 output) and of the gated feed-forward block.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at the end) or, where
`own` is true, through the library's entry points moe_rmsnorm_fwd, moe_rmsnorm_bwd, moe_ffn_fwd and moe_ffn_bwd.
`exact` computes the same outputs from the definitions in 64 bits.

The operators:

  norm      h = x + residual; rstd = 1 / sqrt(mean(h^2) + eps); y = h * rstd * weight, in bf16 and (where the case
            asks for it) also in MXFP8: e4m3 elements with one power-of-two scale per 1x32 block.
  norm_bwd  the gradient of that norm for an upstream dy of y and dh of h, given h, weight and rstd:
            dx = dh + rstd * (weight dy - xhat mean(weight dy xhat)), xhat = h rstd; dweight = sum_t dy xhat.
  ffn       y = W_d (silu(W_g x) * (W_u x)). bf16; or MXFP8, where x (on the way, unless it comes as codes) and the
            activation are quantised to MXFP8 like the weights.
  ffn_step  the bf16 block forward and backward: y, and dx, dW_g, dW_u, dW_d for an upstream dy.
"""
import torch

own = False

EPS = 1e-5
BF = torch.bfloat16


def listed():
    return [
        # one token of a decoding step: residual stream in, normed bf16 for a router and MXFP8 for the experts out
        {"name": "norm decode", "op": "norm", "T": 1, "H": 4096, "residual": True, "mx": True},
        # a prompt or training batch at the width of the MXFP8 configuration, all outputs
        {"name": "norm batch mxfp8", "op": "norm", "T": 8192, "H": 7168, "residual": True, "mx": True},
        # the backward of a training batch, with the residual stream's gradient joined
        {"name": "norm backward batch", "op": "norm_bwd", "T": 8192, "H": 4096, "dh": True},
        # a ragged packed batch at a width that no tile divides, the first norm of a stack (nothing joins h)
        {"name": "norm backward odd", "op": "norm_bwd", "T": 777, "H": 2056, "dh": False},
        # one token of a decoding step: the weights are streamed once
        {"name": "ffn decode", "op": "ffn", "T": 1, "H": 4096, "F": 14336, "mx": False, "codes": False},
        # a decoding batch
        {"name": "ffn decode batch", "op": "ffn", "T": 48, "H": 4096, "F": 14336, "mx": False, "codes": False},
        # a short ragged prompt, widths that no tile divides
        {"name": "ffn odd", "op": "ffn", "T": 333, "H": 2056, "F": 5464, "mx": False, "codes": False},
        # a prompt
        {"name": "ffn prompt", "op": "ffn", "T": 4096, "H": 4096, "F": 14336, "mx": False, "codes": False},
        # the shared expert of the MXFP8 configuration in a decoding step of eight sequences
        {"name": "ffn decode mxfp8", "op": "ffn", "T": 8, "H": 7168, "F": 2048, "mx": True, "codes": False},
        # the same block over a prompt whose norm left it in MXFP8
        {"name": "ffn prompt mxfp8", "op": "ffn", "T": 8192, "H": 7168, "F": 2048, "mx": True, "codes": True},
        # a training step of the dense block
        {"name": "ffn step", "op": "ffn_step", "T": 4096, "H": 4096, "F": 14336},
        # a ragged training step of a small block
        {"name": "ffn step odd", "op": "ffn_step", "T": 1001, "H": 2056, "F": 1544},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ffn", "ffn", "ffn", "ffn_step"])
    if op == "norm":
        mx = rng.random() < 0.6
        step = 32 if mx else 8
        return {"op": op, "T": _log(rng, 1, 8192), "H": step * _log(rng, 512 // step, 7168 // step),
                "residual": rng.random() < 0.7, "mx": mx}
    if op == "norm_bwd":
        return {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 64, 512), "dh": rng.random() < 0.7}
    if op == "ffn":
        if rng.random() < 0.4:
            return {"op": op, "T": _log(rng, 1, 8192), "H": 256 * _log(rng, 4, 28), "F": 128 * _log(rng, 8, 16),
                    "mx": True, "codes": rng.random() < 0.5}
        return {"op": op, "T": _log(rng, 1, 4096), "H": 8 * _log(rng, 128, 512), "F": 8 * _log(rng, 128, 1792),
                "mx": False, "codes": False}
    return {"op": op, "T": _log(rng, 64, 4096), "H": 8 * _log(rng, 128, 512), "F": 8 * _log(rng, 128, 1792)}


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, std):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(BF)


def _tokens(gen, T, H):
    """Hidden states: unit normal, one channel in 64 eight times as large, as residual streams have them."""
    x = torch.randn((T, H), generator=gen, device="cuda", dtype=torch.float32)
    x[:, 5::64] *= 8.0
    return x.to(BF)


def _pow2(e):
    """2^e in fp32, exactly, from its bits (e whole, -126..127; -127, the scale of a block of zeros, gives 0)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _mx(v):
    """(e4m3 codes, scale bytes) of fp32 values in 1x32 blocks along the last dimension: the scale byte is
    floor(log2 amax) - 8 + 127, kept in 0..254 (0 for a block of zeros); elements are rounded to nearest even and
    saturated at 448."""
    b = v.reshape(v.shape[:-1] + (v.shape[-1] // 32, 32))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1
    s = torch.where(amax > 0, (e - 8 + 127).clamp(0, 254), torch.zeros_like(e))
    q = (b * _pow2(127 - s).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(v.shape), s.to(torch.uint8)


def _mx_values(q, s, dtype=torch.float32):
    """The values that codes and scale bytes stand for."""
    b = q.to(dtype).reshape(q.shape[:-1] + (q.shape[-1] // 32, 32))
    return (b * _pow2(s.to(torch.int32) - 127).to(dtype).unsqueeze(-1)).reshape(q.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, T, H = case["op"], case["T"], case["H"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        s["weight"] = (1.0 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(BF)
        if op == "norm":
            s["x"] = _normal(gen, (T, H), 0.5)
            s["residual"] = _tokens(gen, T, H) if case["residual"] else None
        else:
            s["h"] = _tokens(gen, T, H)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
            s["dy"] = _normal(gen, (T, H), 1.0)
            s["dh"] = _normal(gen, (T, H), 1.0) if case["dh"] else None
        return s
    F = case["F"]
    s["x"] = _tokens(gen, T, H)
    W = {"W_g": _normal(gen, (F, H), 0.02), "W_u": _normal(gen, (F, H), 0.02), "W_d": _normal(gen, (H, F), 0.02)}
    for name, w in W.items():
        if case.get("mx"):
            s[name], s[name + "_sf"] = _mx(w.float())
        else:
            s[name] = w
    if case.get("codes"):
        s["x"], s["x_sf"] = _mx(s["x"].float())
    if op == "ffn_step":
        s["dy"] = _normal(gen, (T, H), 1.0)
    return s


# ---------------------------------------------------------------- plain forms

def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        h = s["x"].float()
        if s["residual"] is not None:
            h = h + s["residual"].float()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS)
        y = h * rstd.unsqueeze(-1) * s["weight"].float()
        out = {"h": h.to(BF), "y": y.to(BF), "rstd": rstd}
        if case["mx"]:
            q, sf = _mx(y)
            out["q"], out["sf"] = q, sf.view(torch.float8_e8m0fnu)
        return out
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(-1)
        xhat = s["h"].float() * rstd
        g = dy * s["weight"].float()
        dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(BF), "dweight": (dy * xhat).sum(0, dtype=torch.float64).float()}
    if case.get("mx"):
        x = _mx_values(s["x"], s["x_sf"]) if case["codes"] else _mx_values(*_mx(s["x"].float()))
        Wg, Wu, Wd = (_mx_values(s[n], s[n + "_sf"]) for n in ("W_g", "W_u", "W_d"))
    else:
        x, Wg, Wu, Wd = (s[n].float() for n in ("x", "W_g", "W_u", "W_d"))
    g, u = x @ Wg.t(), x @ Wu.t()
    sg = 1.0 / (1.0 + torch.exp(-g))
    a = g * sg * u
    if case.get("mx"):
        a = _mx_values(*_mx(a))
    y = (a @ Wd.t()).to(BF)
    if op == "ffn":
        return {"y": y}
    dy = s["dy"].float()
    v = dy @ Wd
    dg = v * u * sg * (1.0 + g * (1.0 - sg))
    du = v * g * sg
    return {"y": y, "dx": (dg @ Wg + du @ Wu).to(BF), "dW_g": (dg.t() @ x).to(BF), "dW_u": (du.t() @ x).to(BF),
            "dW_d": (dy.t() @ a).to(BF)}


# ---------------------------------------------------------------- the library's calls

def _plan(s):
    """What a program makes once for its shapes: configuration, output buffers, workspaces."""
    import mixture_experts_layer_aux_b200 as moe
    case = s["case"]
    op, T, H = case["op"], case["T"], case["H"]
    new = lambda *shape, dtype=BF: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    p = {"moe": moe}
    if op == "norm":
        p["out"] = {"h": new(T, H), "y": new(T, H), "rstd": new(T, dtype=torch.float32)}
        p["q"] = p["sf"] = None
        if case["mx"]:
            p["q"], p["sf"] = new(T, H, dtype=torch.uint8), new(T, H // 32, dtype=torch.uint8)
            p["out"]["q"], p["out"]["sf"] = p["q"].view(torch.float8_e4m3fn), p["sf"].view(torch.float8_e8m0fnu)
    elif op == "norm_bwd":
        p["out"] = {"dx": new(T, H), "dweight": new(H, dtype=torch.float32)}
        p["ws"] = moe.workspace(moe.moe_rmsnorm_bwd_workspace_size(T, H))
    else:
        F = case["F"]
        p["cfg"] = moe.make_ffn_config(T=T, H=H, F=F, dtype="mxfp8" if case.get("mx") else "bf16",
                                       save_for_bwd=int(op == "ffn_step"))
        p["ws"] = moe.workspace(moe.moe_ffn_workspace_size(p["cfg"]))
        p["out"] = {"y": new(T, H)}
        if op == "ffn_step":
            p["saved"] = moe.workspace(moe.moe_ffn_saved_size(p["cfg"]))
            p["bwd_ws"] = moe.workspace(moe.moe_ffn_bwd_workspace_size(p["cfg"]))
            p["out"].update(dx=new(T, H), dW_g=new(F, H), dW_u=new(F, H), dW_d=new(H, F))
        byte = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
        p["in"] = {n: byte(s[n]) for n in ("x", "W_g", "W_u", "W_d")}
    return p


def _library(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, op = s["plan"], s["case"]["op"]
    moe, out = p["moe"], p["out"]
    if op == "norm":
        moe.moe_rmsnorm_fwd(s["x"], s["residual"], s["weight"], EPS, out["h"], out["y"], p["q"], p["sf"], out["rstd"])
    elif op == "norm_bwd":
        moe.moe_rmsnorm_bwd(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"], out["dx"], out["dweight"], p["ws"])
    else:
        t = p["in"]
        moe.moe_ffn_fwd(p["cfg"], t["x"], s.get("x_sf"), t["W_g"], t["W_u"], t["W_d"], s.get("W_g_sf"),
                        s.get("W_u_sf"), s.get("W_d_sf"), out["y"], p.get("saved"), p["ws"])
        if op == "ffn_step":
            moe.moe_ffn_bwd(p["cfg"], s["dy"], t["x"], t["W_g"], t["W_u"], t["W_d"], p["saved"], out["dx"],
                            out["dW_g"], out["dW_u"], out["dW_d"], p["bwd_ws"])
    return out


def run(state):
    if own:
        return _library(state)
    return _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, T, H = case["op"], case["T"], case["H"]
    if op == "norm":
        n = 2 + 2 * case["residual"] + 2 + 2 + (1 + 1 / 32) * case["mx"]
        return {"bytes": T * H * n + 2 * H + 4 * T, "flops": 5 * T * H}
    if op == "norm_bwd":
        return {"bytes": T * H * (6 + 2 * case["dh"]) + 6 * H + 4 * T, "flops": 9 * T * H}
    F = case["F"]
    if op == "ffn":
        if case["mx"]:
            x = T * H * (33 / 32 if case["codes"] else 2)
            return {"bytes": 3 * H * F * 33 / 32 + x + 2 * T * H, "flops": 6 * T * H * F}
        return {"bytes": 6 * H * F + 4 * T * H, "flops": 6 * T * H * F}
    return {"bytes": 12 * H * F + 8 * T * H, "flops": 18 * T * H * F}


# ---------------------------------------------------------------- the definitions in 64 bits

def _two_to(k):
    """2^k in 64 bits, exactly (k whole, held in 64 bits), from its bits."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _mx64(v):
    """MXFP8 of 64-bit values by the format's definition: (element values, scales, values)."""
    b = v.reshape(v.shape[:-1] + (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(amax.clamp_min(2.0 ** -1000)))
    # log2 may be off by one at a power of two
    e = torch.where(_two_to(e) > amax, e - 1, e)
    e = torch.where(_two_to(e + 1) <= amax, e + 1, e)
    k = torch.where(amax > 0, (e - 8).clamp(-127, 127), torch.full_like(e, -127.0))
    scale = _two_to(k)
    t = b / scale
    m = t.abs().clamp_min(2.0 ** -6)
    mag = torch.floor(torch.log2(m))
    mag = torch.where(_two_to(mag) > m, mag - 1, mag)
    mag = torch.where(_two_to(mag + 1) <= m, mag + 1, mag)
    step = _two_to(mag - 3)
    q = (torch.round(t / step) * step).clamp(-448.0, 448.0)
    return q.reshape(v.shape), scale.squeeze(-1), (q * scale).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = lambda t: t.double()  # noqa: E731
    if op == "norm":
        h = d(s["x"]) if s["residual"] is None else d(s["x"]) + d(s["residual"])
        rstd = 1.0 / torch.sqrt((h * h).sum(-1) / case["H"] + EPS)
        y = h * rstd[:, None] * d(s["weight"])[None, :]
        out = {"h": h, "y": y, "rstd": rstd}
        if case["mx"]:
            out["q"], out["sf"], _ = _mx64(y)
        return out
    if op == "norm_bwd":
        r = d(s["rstd"])[:, None]
        xhat = d(s["h"]) * r
        gw = d(s["dy"]) * d(s["weight"])[None, :]
        dot = (gw * xhat).sum(-1, keepdim=True) / case["H"]
        dx = gw * r - xhat * r * dot
        if s["dh"] is not None:
            dx = dx + d(s["dh"])
        return {"dx": dx, "dweight": torch.einsum("th,th->h", d(s["dy"]), xhat)}

    def operand(name):
        if name + "_sf" not in s:
            return d(s[name])
        q, sf = s[name], s[name + "_sf"]
        return (d(q).reshape(sf.shape + (32,)) * _two_to(d(sf) - 127.0)[..., None]).reshape(q.shape)

    x, Wg, Wu, Wd = (operand(n) for n in ("x", "W_g", "W_u", "W_d"))
    if case.get("mx") and not case["codes"]:
        x = _mx64(x)[2]
    g = torch.matmul(x, Wg.T)
    u = torch.matmul(x, Wu.T)
    z = torch.sigmoid(g)
    act = g * z * u
    if case.get("mx"):
        act = _mx64(act)[2]
    out = {"y": torch.matmul(act, Wd.T)}
    if op == "ffn_step":
        dy = d(s["dy"])
        da = torch.matmul(dy, Wd)
        dgate = da * u * (z + g * z * (1.0 - z))
        dup = da * (g * z)
        out["dx"] = torch.matmul(dgate, Wg) + torch.matmul(dup, Wu)
        out["dW_g"] = torch.matmul(dgate.T, x)
        out["dW_u"] = torch.matmul(dup.T, x)
        out["dW_d"] = torch.matmul(dy.T, act)
    return out
