"""What a training step of the MoE block keeps in 8 bits, and the norm before it, measured.

Four operators around the experts: the norm whose output the first expert
product reads (`moe_layer_norm`, with its output's codes and an 8-bit
checkpoint of the normalised rows from the same pass), its backward from the
rows or from that checkpoint (`moe_layer_norm_backward`), the experts' FFN that
keeps its pre-activations in 8 bits (`moe_grouped_ffn_fp8_ckpt`), and the
SwiGLU backward from them with every operand the gradient products read
(`moe_swiglu_backward_ckpt`).

`own = False` computes each in elementary torch operations in 32 bits;
`own = True` calls the framework.  E4M3 codes are returned as float8 values
beside their scales.
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # the norm before the layer for one decoded token of the large model: latency counts
        dict(name="norm_token", op="norm", rows=1, cols=7168, bits=16, center=False, bias=False, train=False,
             codes=False),
        # a training batch of the large layer: statistics, the experts' operand in codes, the 8-bit checkpoint
        dict(name="norm_batch", op="norm", rows=8192, cols=7168, bits=16, center=False, bias=False, train=True,
             codes=True),
        # layer norm with a bias of an odd hidden size in fp32 (no whole vectors, ragged batch)
        dict(name="norm_odd_fp32", op="norm", rows=4093, cols=1999, bits=32, center=True, bias=True, train=True,
             codes=False),
        # the norm's backward of a short sample, from the rows kept in bf16
        dict(name="dnorm_short", op="dnorm", rows=131, cols=2048, bits=16, center=True, bias=True, ckpt=False, add=False),
        # the large layer's batch, from the 8-bit checkpoint, the router's and the residual's gradients joined in
        dict(name="dnorm_batch", op="dnorm", rows=8192, cols=7168, bits=16, center=False, bias=False, ckpt=True, add=True),
        # fp32 rows of an odd hidden size, with the gradient of weight and bias
        dict(name="dnorm_odd_fp32", op="dnorm", rows=4093, cols=1999, bits=32, center=True, bias=True, ckpt=False,
             add=False),
        # the experts of the tiny layer
        dict(name="ffn_tiny", op="ffn", rows=512, d=256, F=512, E=8),
        # the experts of the 64-expert replay layer, uneven, some without rows
        dict(name="ffn_replay", op="ffn", rows=24576, d=2048, F=1408, E=64),
        # the tiny layer's SwiGLU backward: latency counts
        dict(name="dswiglu_tiny", op="dswiglu", rows=512, F=512, E=8, rowwise=True, wgrad=True),
        # experts that are not trained (only the dgrad operand and the gates' gradient), long batch
        dict(name="dswiglu_frozen", op="dswiglu", rows=65536, F=2048, E=256, rowwise=True, wgrad=False),
        # every operand of the gradients, the 64-expert replay layer
        dict(name="dswiglu_replay", op="dswiglu", rows=24576, F=1408, E=64, rowwise=True, wgrad=True),
        # every operand of the gradients, the large layer
        dict(name="dswiglu_large", op="dswiglu", rows=65536, F=2048, E=256, rowwise=True, wgrad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "dnorm", "norm", "dnorm", "ffn", "dswiglu", "dswiglu"])
    if op in ("norm", "dnorm"):
        bits = rng.choice([16, 16, 32])
        eight = rng.random() < 0.5                        # whole 128-blocks, so that codes can be asked for
        cols = 128 * _log_int(rng, 1, 64) if eight else _log_int(rng, 16, 8192)
        rows = min(_log_int(rng, 1, 16384), 8192 * 7168 * 2 // (cols * bits // 8))
        c = dict(op=op, rows=rows, cols=cols, bits=bits, center=rng.random() < 0.6, bias=rng.random() < 0.5)
        if op == "norm":
            c.update(train=rng.random() < 0.7, codes=eight and rng.random() < 0.7)
        else:
            c.update(ckpt=eight and rng.random() < 0.6, add=rng.random() < 0.5)
        return c
    E = rng.choice([1, 8, 16, 37, 64])
    if op == "ffn":
        return dict(op=op, rows=_log_int(rng, 1, 16384), d=128 * _log_int(rng, 1, 16), F=128 * _log_int(rng, 1, 11), E=E)
    wgrad = rng.random() < 0.6
    return dict(op=op, rows=_log_int(rng, 1, 65536), F=128 * _log_int(rng, 1, 16), E=E,
                rowwise=not wgrad or rng.random() < 0.7, wgrad=wgrad)


# ---------------------------------------------------------------- the inputs

EPS = 1e-5


def _counts(rows, E):
    """Rows of each expert: uneven, and where there are many experts one in eight without any."""
    p = (1.0 + (torch.arange(E, dtype=torch.float64) * 37) % max(E, 1)).pow(-0.6)
    if E >= 8:
        p[3::8] = 0
    c = torch.floor(p / p.sum() * rows).long()
    c[int(p.argmax())] += rows - int(c.sum())
    return c


def _quant(v):
    """1 x 128 blocks of the last axis: E4M3 values (float8) and fp32 scales amax / 448 (1 where that is 0)."""
    b = v.float().unflatten(-1, (-1, 128))
    s = b.abs().amax(-1) / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (b / s[..., None]).flatten(-2).to(F8), s


def _deq(q, s):
    return (q.float().unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *n: torch.randn(*n, device=DEV, generator=g)  # noqa: E731
    s = dict(case=case, keep={})
    op = case["op"]
    if op in ("norm", "dnorm"):
        R, C = case["rows"], case["cols"]
        dt = torch.bfloat16 if case["bits"] == 16 else torch.float32
        # a residual stream: rows of different size and offset, a few channels far larger than the rest
        ch = torch.where(torch.rand(C, device=DEV, generator=g) < 0.01, 12.0, 1.0)
        x = (r(R, C) * ch + 0.3 * r(R, 1)) * (0.3 + 3 * torch.rand(R, 1, device=DEV, generator=g))
        s["x"] = x.to(dt)
        s["w"] = (1.0 + 0.2 * r(C)).to(dt)
        s["b"] = (0.1 * r(C)).to(dt) if case["bias"] else None
        if op == "norm":
            return s
        xf = s["x"].double()
        mu = xf.mean(1, keepdim=True) if case["center"] else torch.zeros(R, 1, dtype=torch.float64, device=DEV)
        rs = ((xf - mu).square().mean(1, keepdim=True) + EPS).rsqrt()
        s["mean"], s["rstd"] = mu[:, 0].float(), rs[:, 0].float()
        if case["ckpt"]:
            q, sc = _quant((xf - mu) * rs)
            s["ckpt"] = (q.view(torch.uint8), sc)
            s["x"] = None
        s["dy"] = (1e-3 * r(R, C)).to(dt)
        s["dy_add"] = 1e-4 * r(R, C) if case["add"] else None
        s["dx_add"] = (1e-3 * r(R, C)).to(dt) if case["add"] else None
        return s
    A, F, E = case["rows"], case["F"], case["E"]
    cnt = _counts(A, E)
    zero = torch.zeros(1, dtype=torch.int64)
    off = torch.cat([zero, cnt.cumsum(0)])
    s["offsets"] = off.int().to(DEV)
    if op == "ffn":
        d = case["d"]
        s["cap"] = int(cnt.max())                         # the most rows of an expert, as the dispatch's plan has it
        q, s["xs"] = _quant(r(A, d) * (0.5 + torch.rand(A, 1, device=DEV, generator=g)))
        s["xq"] = q.view(torch.uint8)
        for n, N, K in (("w13", 2 * F, d), ("w2", d, F)):
            b = (0.02 * r(E, N, K)).unflatten(2, (-1, 128)).unflatten(1, (-1, 128))
            sc = b.abs().amax((2, 4)) / 448.0
            s[n + "q"] = (b / sc[:, :, None, :, None]).flatten(3, 4).flatten(1, 2).to(F8).view(torch.uint8)
            s[n + "s"] = sc
        return s
    s["dact"] = (1e-3 * r(A, F) * (0.2 + torch.rand(A, 1, device=DEV, generator=g))).bfloat16()
    q, s["hs"] = _quant(1.2 * r(A, 2 * F) * (0.5 + torch.rand(A, 1, device=DEV, generator=g)))
    s["hq"] = q.view(torch.uint8)
    s["gates"] = 0.05 + torch.rand(A, device=DEV, generator=g)
    s["sl2"] = torch.randperm(A, device=DEV, generator=g).int()       # where each slot's row was sorted to
    if case["wgrad"]:
        pad = torch.cat([zero, ((cnt + 127) // 128 * 128).cumsum(0)])
        s["pad"], s["ld"] = pad.int().to(DEV), int(pad[-1])
    return s


# ------------------------------------------------------------ the operators

def run(s):
    op = s["case"]["op"]
    return (OWN if own else PLAIN)[op](s)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    mean = x.mean(1, keepdim=True) if c["center"] else None
    xc = x - mean if c["center"] else x
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
    xhat = xc * rstd
    y = xhat * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = {"y": y.to(s["x"].dtype)}
    if c["train"]:
        out["rstd"] = rstd[:, 0]
        if c["center"]:
            out["mean"] = mean[:, 0]
    if c["codes"]:
        out["y_q"], out["y_s"] = _quant(y)
        out["xhat_q"], out["xhat_s"] = _quant(xhat)
    return out


def _plain_dnorm(s):
    c = s["case"]
    rs = s["rstd"][:, None]
    if c["ckpt"]:
        xhat = _deq(s["ckpt"][0].view(F8), s["ckpt"][1])
    else:
        xhat = s["x"].float()
        xhat = (xhat - s["mean"][:, None] if c["center"] else xhat) * rs
    dy = s["dy"].float()
    if c["add"]:
        dy = dy + s["dy_add"]
    g = dy * s["w"].float()
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if c["center"]:
        d = d - g.mean(1, keepdim=True)
    d = d * rs
    if c["add"]:
        d = d + s["dx_add"].float()
    out = {"dx": d.to(s["dy"].dtype), "dw": (dy * xhat).sum(0)}
    if c["bias"]:
        out["db"] = dy.sum(0)
    return out


def _plain_ffn(s):
    c = s["case"]
    off = s["offsets"].long()
    A, F, E = c["rows"], c["F"], c["E"]
    row = torch.arange(A, device=DEV)
    e = torch.searchsorted(off[1:], row, right=True)
    at = e * s["cap"] + row - off[e]                      # each expert's rows in a block of its own
    spread = lambda v: v.new_zeros(E * s["cap"], v.shape[1]).index_copy_(0, at, v).view(E, s["cap"], -1)  # noqa: E731
    deq_w = lambda q, sc: (q.view(F8).float().unflatten(2, (-1, 128)).unflatten(1, (-1, 128)) *  # noqa: E731
                           sc[:, :, None, :, None]).flatten(3, 4).flatten(1, 2)
    h = torch.bmm(spread(_deq(s["xq"].view(F8), s["xs"])), deq_w(s["w13q"], s["w13s"]).transpose(1, 2)).flatten(0, 1)[at]
    h_q, h_s = _quant(h)
    gate, up = h[:, :F], h[:, F:]
    act = gate / (1.0 + torch.exp(-gate)) * up
    a_q, a_s = _quant(act)
    out = torch.bmm(spread(_deq(a_q, a_s)), deq_w(s["w2q"], s["w2s"]).transpose(1, 2)).flatten(0, 1)[at]
    return {"out": out.bfloat16(), "h_q": h_q, "h_s": h_s}


def _plain_dswiglu(s):
    c = s["case"]
    F, E = c["F"], c["E"]
    h = _deq(s["hq"].view(F8), s["hs"])
    gate, up = h[:, :F], h[:, F:]
    a = s["dact"].float()
    sg = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sg * up
    dh = torch.cat([a * up * sg * (1.0 + gate * (1.0 - sg)), a * gate * sg], 1)
    out = {"d_gates": (a * act).sum(1)[s["sl2"].long()] / s["gates"]}
    if c["rowwise"]:
        out["dh_q"], out["dh_s"] = _quant(dh)
    if c["wgrad"]:
        off, pad, ld = s["offsets"].long(), s["pad"].long(), s["ld"]
        at = torch.arange(ld, device=DEV)
        e = torch.searchsorted(pad[1:], at, right=True).clamp_max(E - 1)
        src = off[e] + at - pad[e]
        live = (src < off[e + 1])[:, None]
        src = src.clamp_max(max(c["rows"] - 1, 0))
        for_wgrad = lambda v: torch.where(live, v[src], 0.0).t().contiguous()  # noqa: E731
        q, sc = _quant(for_wgrad(dh))
        out["dhT_q"], out["dhT_s"] = q, sc.t().contiguous()
        q, sc = _quant(for_wgrad(act))
        out["actT_q"], out["actT_s"] = q, sc.t().contiguous()
    return out


PLAIN = dict(norm=_plain_norm, dnorm=_plain_dnorm, ffn=_plain_ffn, dswiglu=_plain_dswiglu)


def _keep(s, size):
    """The workspace a program keeps beside its plan, made on the first pass."""
    if "ws" not in s["keep"]:
        s["keep"]["ws"] = torch.empty(max(256, size()), dtype=torch.uint8, device=DEV)
    return s["keep"]["ws"]


def _own_norm(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    y, mean, rstd, codes, ckpt = L.moe_layer_norm(s["x"], s["w"], s["b"], eps=EPS, center=c["center"],
                                                  mean=c["train"] and c["center"], rstd=c["train"], codes=c["codes"],
                                                  ckpt=c["codes"])
    out = {"y": y}
    if c["train"]:
        out["rstd"] = rstd
        if c["center"]:
            out["mean"] = mean
    if c["codes"]:
        out["y_q"], out["y_s"] = codes[0].view(F8), codes[1]
        out["xhat_q"], out["xhat_s"] = ckpt[0].view(F8), ckpt[1]
    return out


def _own_dnorm(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_layer_norm_backward_workspace_size(c["rows"], c["cols"]))
    dx, dw, db = L.moe_layer_norm_backward(s["dy"], s["rstd"], x=s["x"], mean=s["mean"] if c["center"] else None,
                                           ckpt=s["ckpt"] if c["ckpt"] else None, weight=s["w"], center=c["center"],
                                           dy_add=s["dy_add"], dx_add=s["dx_add"], dbias=c["bias"], workspace=ws)
    out = {"dx": dx, "dw": dw}
    if c["bias"]:
        out["db"] = db
    return out


def _own_ffn(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_grouped_ffn_workspace_size(c["rows"], c["d"], c["F"]))
    out, h_q, h_s = L.moe_grouped_ffn_fp8_ckpt(s["xq"], s["xs"], s["offsets"], s["w13q"], s["w13s"], s["w2q"],
                                               s["w2s"], workspace=ws)
    return {"out": out, "h_q": h_q.view(F8), "h_s": h_s}


def _own_dswiglu(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_swiglu_backward_ckpt_workspace_size(c["rows"], c["F"]))
    kw = dict(expert_offsets=s["offsets"], pad=s["pad"], ld=s["ld"], dhT=True, actT=True) if c["wgrad"] else {}
    dh, d_gates, dhT, actT = L.moe_swiglu_backward_ckpt(s["dact"], s["hq"], s["hs"], gates=s["gates"],
                                                        slot_to_sorted=s["sl2"], dh=c["rowwise"], d_gates=True,
                                                        workspace=ws, **kw)
    out = {"d_gates": d_gates}
    if c["rowwise"]:
        out["dh_q"], out["dh_s"] = dh[0].view(F8), dh[1]
    if c["wgrad"]:
        out["dhT_q"], out["dhT_s"] = dhT[0].view(F8), dhT[1]
        out["actT_q"], out["actT_s"] = actT[0].view(F8), actT[1]
    return out


OWN = dict(norm=_own_norm, dnorm=_own_dnorm, ffn=_own_ffn, dswiglu=_own_dswiglu)


# ----------------------------------------------------------- what it cannot do without

def work(case):
    op = case["op"]
    eight = 1 + 4 / 128                                    # a code and its share of the block's scale
    if op in ("norm", "dnorm"):
        n, b = case["rows"] * case["cols"], case["bits"] // 8
        if op == "norm":
            stats = 4 * case["rows"] * (case["train"] * (1 + case["center"]))
            return {"bytes": n * (2 * b + (2 * eight if case["codes"] else 0)) + stats +
                    case["cols"] * b * (1 + case["bias"]), "flops": 8 * n}
        per = 2 * b + (eight if case["ckpt"] else b) + ((4 + b) if case["add"] else 0)
        return {"bytes": n * per + case["rows"] * (8 if case["center"] and not case["ckpt"] else 4) +
                case["cols"] * (b + 4 * (1 + case["bias"])), "flops": 14 * n}
    A, F, E = case["rows"], case["F"], case["E"]
    if op == "ffn":
        d = case["d"]
        used = int((_counts(A, E) > 0).sum())
        return {"bytes": A * (d * eight + 2 * F * eight + 2 * d) + used * 3 * d * F * (1 + 4 / 16384) + 4 * (E + 1),
                "flops": 6 * A * d * F}
    b = A * F * (2 + 2 * eight) + 12 * A + (A * 2 * F * eight if case["rowwise"] else 0)
    if case["wgrad"]:
        b += 3 * F * int(((_counts(A, E) + 127) // 128 * 128).sum()) * eight + 8 * (E + 1)
    return {"bytes": b, "flops": 25 * A * F}


# ------------------------------------------------------------------ in 64 bits

def _code64(v, axis):
    """E4M3 nearest-even of v / (amax / 448) over runs of 128 along `axis`, in 64 bits: values and scales."""
    t = v.movedim(axis, -1)
    t = t.reshape(*t.shape[:-1], t.shape[-1] // 128, 128)
    sc = t.abs().amax(-1) / 448.0
    sc = torch.where(sc == 0, torch.ones_like(sc), sc)
    z = t / sc[..., None]
    step = torch.exp2(torch.clamp_min(torch.frexp(z).exponent.double() - 1, -6.0) - 3.0)
    z = (torch.round(z / step) * step).clamp(-448.0, 448.0)
    return z.reshape(*z.shape[:-2], -1).movedim(-1, axis), sc.movedim(-1, axis)


def _val64(q, sc, axis=1):
    return q.view(F8).double() * sc.double().repeat_interleave(128, axis)


def _exact_norm(case, s):
    x, w = s["x"].double(), s["w"].double()
    var, mu = torch.var_mean(x, 1, correction=0, keepdim=True)
    if not case["center"]:
        var, mu = var + mu * mu, torch.zeros_like(mu)
    rstd = 1.0 / torch.sqrt(var + EPS)
    xhat = (x - mu) * rstd
    y = torch.addcmul(torch.zeros_like(w) if s["b"] is None else s["b"].double(), xhat, w)
    out = {"y": y}
    if case["train"]:
        out["rstd"] = rstd.flatten()
        if case["center"]:
            out["mean"] = mu.flatten()
    if case["codes"]:
        out["y_q"], out["y_s"] = _code64(y, 1)
        out["xhat_q"], out["xhat_s"] = _code64(xhat, 1)
    return out


def _exact_dnorm(case, s):
    rs = s["rstd"].double()[:, None]
    if case["ckpt"]:
        xhat = _val64(*s["ckpt"])
    else:
        xhat = s["x"].double()
        xhat = rs * (xhat - s["mean"].double()[:, None]) if case["center"] else rs * xhat
    dy = s["dy"].double()
    if case["add"]:
        dy += s["dy_add"].double()
    out = {"dw": torch.einsum("rc,rc->c", dy, xhat)}
    if case["bias"]:
        out["db"] = dy.sum(0)
    dy *= s["w"].double()
    n = dy.shape[1]
    m2 = torch.einsum("rc,rc->r", dy, xhat)[:, None] / n
    m1 = dy.sum(1, keepdim=True) / n if case["center"] else 0.0
    dx = rs * (dy - m1 - m2 * xhat)
    out["dx"] = dx + s["dx_add"].double() if case["add"] else dx
    return out


def _exact_ffn(case, s):
    A, F = case["rows"], case["F"]
    if 6 * A * case["d"] * F > 5e12:
        return None
    cuts = s["offsets"].tolist()
    x = _val64(s["xq"], s["xs"])
    h = x.new_empty(A, 2 * F)
    out = x.new_empty(A, case["d"])
    for e in range(case["E"]):
        r = slice(cuts[e], cuts[e + 1])
        if cuts[e] == cuts[e + 1]:
            continue
        w13 = _val64(s["w13q"][e], s["w13s"][e].repeat_interleave(128, 0))
        w2 = _val64(s["w2q"][e], s["w2s"][e].repeat_interleave(128, 0))
        h[r] = x[r] @ w13.t()
        act = h[r, F:] * h[r, :F] * torch.sigmoid(h[r, :F])
        z, sc = _code64(act, 1)
        out[r] = (z * sc.repeat_interleave(128, 1)) @ w2.t()
    h_q, h_s = _code64(h, 1)
    return {"out": out, "h_q": h_q, "h_s": h_s}


def _exact_dswiglu(case, s):
    A, F, E = case["rows"], case["F"], case["E"]
    h = _val64(s["hq"], s["hs"])
    a = s["dact"].double()
    g, u = h[:, :F], h[:, F:]
    sg = torch.sigmoid(g)
    dh = torch.empty_like(h)
    dh[:, :F] = a * u * (sg + g * sg * torch.sigmoid(-g))
    dh[:, F:] = a * g * sg
    dg = (dh[:, F:] * u).sum(1)
    out = {"d_gates": dg[s["sl2"].long()] / s["gates"].double()}
    if case["rowwise"]:
        out["dh_q"], out["dh_s"] = _code64(dh, 1)
    if case["wgrad"]:
        cuts, pads = s["offsets"].tolist(), s["pad"].tolist()
        for name, v in (("dhT", dh), ("actT", g * sg * u)):
            t = v.new_zeros(s["ld"], v.shape[1])
            for e in range(E):
                t[pads[e]:pads[e] + cuts[e + 1] - cuts[e]] = v[cuts[e]:cuts[e + 1]]
            q, sc = _code64(t, 0)
            out[name + "_q"], out[name + "_s"] = q.t().contiguous(), sc.contiguous()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, dnorm=_exact_dnorm, ffn=_exact_ffn, dswiglu=_exact_dswiglu)[case["op"]](case, s)
