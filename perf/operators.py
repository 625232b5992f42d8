"""The router's and the policy's losses of one RL training step, measured.

Five operators that a trainer calls around the MoE layer: log-probabilities of
sampled tokens (`moe_token_logprobs`), the clipped policy loss with a KL term
and its gradient (`moe_policy_loss`), every expert's router logit
(`moe_router_logits`), the balance and z losses with per-expert counts and the
gradient of the logits (`moe_balance_loss`), and the router's gradients from
dense logit gradients (`moe_router_backward_dense`).

`own = False` computes each in elementary torch operations in 32 bits (sums of
a whole batch in 64); `own = True` calls the framework.
"""
import math

import torch

own = False

SOFTMAX, SIGMOID = 0, 1
DEV = "cuda"


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # log-probs of a full packed micro-batch under the frozen reference policy (half precision, large vocabulary)
        dict(name="logprobs_batch", op="logprobs", N=8192, V=131072, bits=16, prompt=0, tau=1.0),
        # log-probs of a handful of sampled tokens, fp32 logits, odd vocabulary: latency counts
        dict(name="logprobs_few", op="logprobs", N=7, V=50001, bits=32, prompt=0, tau=0.8),
        # policy update of a short sample: few rows, an eighth of them prompt
        dict(name="policy_short", op="policy", N=256, V=32768, bits=16, prompt=16, tau=1.0, ref=True, eta=0.0),
        # policy update with fp32 logits, an odd vocabulary and an entropy bonus
        dict(name="policy_fp32_odd", op="policy", N=1021, V=65537, bits=32, prompt=32, tau=0.7, ref=True, eta=0.01),
        # policy update of a full packed micro-batch, a quarter of its tokens prompt (masked)
        dict(name="policy_batch", op="policy", N=8192, V=131072, bits=16, prompt=32, tau=1.0, ref=True, eta=0.0),
        # every expert's logit of a ragged batch on the 64-expert replay layer
        dict(name="logits_e64_ragged", op="logits", T=4093, d=2048, E=64),
        # every expert's logit of the large layer (replay computes only the chosen ones)
        dict(name="logits_large", op="logits", T=8192, d=7168, E=256),
        # balance loss of the tiny layer: latency counts
        dict(name="balance_tiny", op="balance", T=256, E=8, k=2, score=SOFTMAX, seqs=1, mask=False, gates=False),
        # balance + z loss of the large layer with the gates' gradients (sigmoid scores, renormalised gates)
        dict(name="balance_large", op="balance", T=8192, E=256, k=8, score=SIGMOID, seqs=1, mask=False, gates=True),
        # sequence-wise balance loss of a long packed batch with padding tokens
        dict(name="balance_long_seqs", op="balance", T=131072, E=256, k=8, score=SIGMOID, seqs=24, mask=True,
             gates=True),
        # the router's gradients of a ragged batch on the 64-expert replay layer
        dict(name="rbwd_e64_ragged", op="rbwd", T=4093, d=2048, E=64),
        # the router's gradients of the large layer
        dict(name="rbwd_large", op="rbwd", T=8192, d=7168, E=256),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["logprobs", "policy", "logits", "balance", "rbwd"])
    if op in ("logprobs", "policy"):
        bits = rng.choice([16, 16, 32])
        V = _log_int(rng, 1000, 131072)
        if rng.random() < 0.5:
            V = max(8, V // 8 * 8)
        N = _log_int(rng, 1, 8192 if bits == 16 else 4096)
        prompt = rng.choice([0, 8, 32, 57])
        c = dict(op=op, N=N, V=V if V != 3072 else 3080, bits=bits, prompt=prompt if N > 2 * prompt else 0,
                 tau=rng.choice([1.0, 0.6, 1.3]))
        if op == "policy":
            c.update(ref=rng.random() < 0.6, eta=rng.choice([0.0, 0.0, 0.003]))
        return c
    E = rng.choice([8, 16, 37, 64, 96, 128, 160, 256])
    k = rng.choice([1, 2, 4, 6, 8])
    if op == "balance":
        T = _log_int(rng, 1, 131072)
        seqs = rng.choice([1, 1, 3, 17])
        return dict(op=op, T=T, E=E, k=k, score=rng.choice([SOFTMAX, SIGMOID]), seqs=seqs if T > 64 else 1,
                    mask=T > 64 and rng.random() < 0.5, gates=rng.random() < 0.7)
    d = 128 * _log_int(rng, 1, 56)
    return dict(op=op, T=_log_int(rng, 1, 8192), d=d if d != 3072 else 3200, E=E)


# ---------------------------------------------------------------- the inputs

SEG = 128   # tokens of one packed sample; its first `prompt` tokens are the prompt (weight 0)


def _active(case):
    full, tail = divmod(case["N"], SEG)
    return full * (SEG - case["prompt"]) + max(0, tail - case["prompt"])


def _token_inputs(case, g):
    N, V = case["N"], case["V"]
    dt = torch.bfloat16 if case["bits"] == 16 else torch.float32
    logits = torch.empty(N, V, dtype=dt, device=DEV)
    targets = torch.empty(N, dtype=torch.int64, device=DEV)
    lp = torch.empty(N, dtype=torch.float64, device=DEV)
    rows = max(1, (1 << 27) // V)
    for r in range(0, N, rows):
        e = min(N, r + rows)
        z = torch.randn(e - r, V, device=DEV, generator=g)
        z = z * (2.0 + 2.0 * torch.rand(e - r, 1, device=DEV, generator=g))      # sharper and flatter rows
        logits[r:e] = z
        z = logits[r:e].float() / case["tau"]
        u = torch.rand(e - r, V, device=DEV, generator=g).clamp_(1e-9, 1 - 1e-7)  # sampled from the policy itself
        targets[r:e] = (z - torch.log(-torch.log(u))).argmax(1)
        lp[r:e] = z.gather(1, targets[r:e, None])[:, 0].double() - torch.logsumexp(z.double(), 1)
    return logits, targets, lp


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case, keep={})
    op = case["op"]
    if op in ("logprobs", "policy"):
        N = case["N"]
        s["logits"], y, lp = _token_inputs(case, g)
        pos = torch.arange(N, device=DEV) % SEG
        live = pos >= case["prompt"]
        if op == "logprobs":
            s["targets"] = torch.where(live, y, -100)          # prompt tokens are not scored
            return s
        s["targets"] = y
        noise = 0.15 * torch.randn(N, device=DEV, generator=g).double()
        for border in (math.log(1 - 0.2), math.log(1 + 0.28)):  # not next to a border of the clipping
            noise = torch.where((noise - border).abs() < 1e-3, noise + 3e-3, noise)
        s["old"] = (lp - noise).float()
        s["ref"] = (lp + 0.1 * torch.randn(N, device=DEV, generator=g).double()).float() if case["ref"] else None
        seg = torch.arange(N, device=DEV) // SEG
        s["adv"] = (0.3 + torch.randn(N // SEG + 1, device=DEV, generator=g))[seg]   # one advantage per sample
        s["w"] = live.float() * (0.5 + torch.rand(N // SEG + 1, device=DEV, generator=g)[seg])
        return s
    T, E = case["T"], case["E"]
    if op == "balance":
        k = case["k"]
        pop = 0.7 * torch.randn(E, device=DEV, generator=g)      # some experts are popular
        s["logits"] = torch.randn(T, E, device=DEV, generator=g) + pop
        s["ids"] = s["logits"].topk(k, 1).indices.int()
        s["mask"] = torch.rand(T, device=DEV, generator=g) < 0.9 if case["mask"] else None
        s["offsets"] = None
        if case["seqs"] > 1:
            cut = torch.randint(0, T + 1, (case["seqs"] - 2,), device=DEV, generator=g).sort().values
            zero, end = cut.new_zeros(2), cut.new_full((1,), T)   # the first sequence is empty
            s["offsets"] = torch.cat([zero, cut, end]).int()
        s["dg"] = 1e-4 * torch.randn(T, k, device=DEV, generator=g) if case["gates"] else None
        return s
    d = case["d"]
    s["x"] = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    s["wr"] = (0.02 * torch.randn(E, d, device=DEV, generator=g)).bfloat16()
    if op == "rbwd":
        # logit gradients: small everywhere, larger at the chosen experts
        s["dl"] = 1e-6 * torch.randn(T, E, device=DEV, generator=g)
        at = torch.randint(0, E, (T, 2), device=DEV, generator=g)
        s["dl"].scatter_add_(1, at, 1e-4 * torch.randn(T, 2, device=DEV, generator=g))
    return s


# ------------------------------------------------------------ the operators

CLIP_LOW, CLIP_HIGH, BETA = 0.2, 0.28, 0.02
ALPHA, ZETA, ROUTE_SCALE = 1e-2, 1e-3, 2.5


def run(s):
    op = s["case"]["op"]
    return (OWN if own else PLAIN)[op](s)


def _plain_rows(s):
    """lp, H, p and log p of every row, fp32; rows that are not scored give zeros."""
    c = s["case"]
    z = s["logits"].float() / c["tau"]
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    logp = z - torch.log(total)
    p = e / total
    ent = -(p * torch.where(p > 0, logp, 0.0)).sum(1)
    ok = s["targets"] >= 0
    lp = logp.gather(1, s["targets"].clamp_min(0)[:, None])[:, 0]
    return torch.where(ok, lp, 0.0), torch.where(ok, ent, 0.0), p, logp


def _plain_logprobs(s):
    lp, ent, _, _ = _plain_rows(s)
    return {"logprobs": lp, "entropy": ent}


def _plain_policy(s):
    c = s["case"]
    lp, ent, p, logp = _plain_rows(s)
    A, w = s["adv"], s["w"]
    r = torch.exp(torch.clamp_max(lp - s["old"], 80.0))
    clipped = torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH)
    pg = torch.maximum(-A * r, -A * clipped)
    off = -A * clipped > -A * r                                # the clipped side: no gradient
    gain = torch.where(off, 0.0, -A * r)
    kl = torch.zeros_like(lp)
    if s["ref"] is not None:
        q = torch.clamp_max(s["ref"].double() - lp.double(), 80.0)
        kl = torch.expm1(q) - q
        gain = gain - BETA * torch.expm1(q).float()
    wd = w.double()
    norm = wd.sum()
    mean = lambda v: (torch.where(w != 0, wd * v.double(), 0.0)).sum() / norm  # noqa: E731
    beta = BETA if s["ref"] is not None else 0.0
    m = [mean(pg), mean(kl), mean(ent), mean(off)]
    loss = m[0] + beta * m[1] - c["eta"] * m[2]
    stats = torch.stack([loss, *m, norm]).float()
    coef = torch.where(w != 0, wd / norm / c["tau"], 0.0).float()[:, None]
    d = -gain[:, None] * p
    if c["eta"]:
        d = d + c["eta"] * p * (torch.where(p > 0, logp, 0.0) + ent[:, None])
    d.scatter_add_(1, s["targets"][:, None], gain[:, None])
    return {"loss": stats[0], "stats": stats, "logprobs": torch.where(w != 0, lp, 0.0),
            "dlogits": (coef * d).to(s["logits"].dtype)}


def _plain_logits(s):
    return {"logits": s["x"].float() @ s["wr"].float().t()}


def _plain_balance(s):
    c = s["case"]
    l, ids = s["logits"], s["ids"].long()
    T, E = l.shape
    k, B = ids.shape[1], c["seqs"]
    mask = torch.ones(T, device=DEV) if s["mask"] is None else s["mask"].float()
    seq = torch.zeros(T, dtype=torch.int64, device=DEV)
    if s["offsets"] is not None:
        seq = torch.searchsorted(s["offsets"][1:].long(), torch.arange(T, device=DEV), right=True)
    hits = torch.zeros(B * E, dtype=torch.float64, device=DEV)
    hits.index_add_(0, (seq[:, None] * E + ids).reshape(-1), mask.double()[:, None].expand(T, k).reshape(-1))
    counts = hits.view(B, E)
    n_b = torch.zeros(B, dtype=torch.float64, device=DEV).index_add_(0, seq, mask.double())
    n = n_b.sum().clamp_min(1.0)
    full = (n_b > 0).double().sum().clamp_min(1.0)
    f = (counts * E / (k * n_b.clamp_min(1.0)[:, None])).float()[seq]              # [T, E]
    share = (mask.double() / (full * n_b.clamp_min(1.0))[seq])
    top = l.amax(1, keepdim=True)
    ex = torch.exp(l - top)
    tot = ex.sum(1, keepdim=True)
    soft, lse = ex / tot, (top + torch.log(tot))[:, 0]
    if c["score"] == SOFTMAX:
        q, slope = soft, soft
    else:
        sg = 1.0 / (1.0 + torch.exp(-l))
        q = sg / sg.sum(1, keepdim=True)
        slope = q / (1.0 + torch.exp(l))
    dot = (f * q).sum(1, keepdim=True)
    losses = torch.stack([ALPHA * (share * dot[:, 0].double()).sum(),
                          ZETA * (mask.double() * lse.double().square()).sum() / n]).float()
    dl = (ALPHA * share).float()[:, None] * slope * (f - dot)
    dl = dl + (2 * ZETA * mask * lse / n.float())[:, None] * soft
    if s["dg"] is not None:
        dg, li = s["dg"], l.gather(1, ids)
        if c["score"] == SOFTMAX:
            p = torch.exp(li - li.amax(1, keepdim=True))
            p = p / p.sum(1, keepdim=True)
            gd = p * (dg - (dg * p).sum(1, keepdim=True))
        else:
            si = 1.0 / (1.0 + torch.exp(-li))
            S = si.sum(1, keepdim=True)
            gd = si / (1.0 + torch.exp(li)) * (dg - (dg * si).sum(1, keepdim=True) / S) / S
        dl = dl.scatter_add(1, ids, ROUTE_SCALE * gd)
    return {"losses": losses, "counts": counts.int(), "d_logits": dl}


def _plain_rbwd(s):
    return {"dx": s["dl"] @ s["wr"].float(), "dw": s["dl"].t() @ s["x"].float()}


PLAIN = dict(logprobs=_plain_logprobs, policy=_plain_policy, logits=_plain_logits, balance=_plain_balance,
             rbwd=_plain_rbwd)


def _keep(s, size):
    """The workspace a program keeps beside its plan, made on the first pass."""
    if "ws" not in s["keep"]:
        s["keep"]["ws"] = torch.empty(max(16, size()), dtype=torch.uint8, device=DEV)
    return s["keep"]["ws"]


def _own_logprobs(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    lp, ent = L.moe_token_logprobs(s["logits"], s["targets"], temperature=s["case"]["tau"], entropy=True)
    return {"logprobs": lp, "entropy": ent}


def _own_policy(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_policy_loss_workspace_size(c["N"], c["V"]))
    stats, lp, dl = L.moe_policy_loss(s["logits"], s["targets"], s["old"], s["adv"], ref_logprobs=s["ref"],
                                      weights=s["w"], temperature=c["tau"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                                      kl_coef=BETA, entropy_coef=c["eta"], workspace=ws)
    return {"loss": stats[0], "stats": stats, "logprobs": lp, "dlogits": dl}


def _own_logits(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_router_logits_workspace_size(c["T"], c["d"], c["E"]))
    return {"logits": L.moe_router_logits(s["x"], s["wr"], workspace=ws)}


def _own_balance(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_balance_loss_workspace_size(c["T"], c["E"], c["seqs"]))
    losses, counts, dl = L.moe_balance_loss(s["logits"], s["ids"], c["score"], ALPHA, z_coef=ZETA,
                                            token_mask=s["mask"], seq_offsets=s["offsets"], d_gates=s["dg"],
                                            route_scale=ROUTE_SCALE, workspace=ws)
    return {"losses": losses, "counts": counts, "d_logits": dl}


def _own_rbwd(s):
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    c = s["case"]
    ws = _keep(s, lambda: L.moe_router_backward_dense_workspace_size(c["T"], c["d"], c["E"]))
    dx, dw = L.moe_router_backward_dense(s["x"], s["wr"], s["dl"], workspace=ws)
    return {"dx": dx, "dw": dw}


OWN = dict(logprobs=_own_logprobs, policy=_own_policy, logits=_own_logits, balance=_own_balance, rbwd=_own_rbwd)


# ----------------------------------------------------------- what it cannot do without

def work(case):
    op = case["op"]
    if op in ("logprobs", "policy"):
        N, V, b = case["N"], case["V"], case["bits"] // 8
        rows = _active(case)
        if op == "logprobs":
            return {"bytes": rows * V * b + 8 * N + 8 * N, "flops": 6 * rows * V}
        return {"bytes": rows * V * b + N * V * b + (8 + 4 * (4 if case["ref"] else 3)) * N + 4 * N + 24,
                "flops": 12 * rows * V}
    T, E = case["T"], case["E"]
    if op == "balance":
        k = case["k"]
        return {"bytes": 8 * T * E + 4 * T * k * (2 if case["gates"] else 1) + (T if case["mask"] else 0) +
                4 * case["seqs"] * E + 8, "flops": 20 * T * E}
    d = case["d"]
    if op == "logits":
        return {"bytes": 2 * T * d + 2 * E * d + 4 * T * E, "flops": 2 * T * d * E}
    return {"bytes": 2 * T * d + 2 * E * d + 4 * T * E + 4 * T * d + 4 * E * d, "flops": 4 * T * d * E}


# ------------------------------------------------------------------ in 64 bits

def _exact_tokens(case, s):
    N, V, tau = case["N"], case["V"], case["tau"]
    y, pol = s["targets"], case["op"] == "policy"
    lps = torch.zeros(N, dtype=torch.float64, device=DEV)
    ents = torch.zeros_like(lps)
    acc = torch.zeros(5, dtype=torch.float64, device=DEV)       # pg, kl, entropy, clipped, weight
    out = torch.zeros(N, V, dtype=torch.float64, device=DEV) if pol else None
    live = (s["w"] != 0) if pol else (y >= 0)
    norm = s["w"].double().sum() if pol else None
    step = max(1, (1 << 26) // V)
    at = torch.nonzero(live)[:, 0]
    for r in range(0, at.numel(), step):
        i = at[r:r + step]
        j = torch.arange(i.numel(), device=DEV)
        z = s["logits"][i].double() / tau
        logp = z - torch.logsumexp(z, 1, keepdim=True)
        p = logp.exp()
        H = -(p * logp).sum(1)
        lp = logp[j, y[i]]
        lps[i], ents[i] = lp, H
        if not pol:
            continue
        A, w = s["adv"][i].double(), s["w"][i].double()
        ratio = (lp - s["old"][i].double()).exp()
        lo, hi = A * ratio, A * ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH)
        gain = torch.where(lo <= hi, -A * ratio, torch.zeros_like(A))
        kl = torch.zeros_like(A)
        if s["ref"] is not None:
            u = s["ref"][i].double() - lp
            kl = u.exp() - u - 1
            gain = gain + BETA * (1 - u.exp())
        acc += torch.stack([(w * -torch.minimum(lo, hi)).sum(), (w * kl).sum(), (w * H).sum(),
                            (w * (lo > hi)).sum(), w.sum()])
        d = case["eta"] * p * (logp + H[:, None]) - gain[:, None] * p
        d[j, y[i]] += gain
        out[i] = d * (w / norm / tau)[:, None]
    if not pol:
        return {"logprobs": lps, "entropy": ents}
    m = acc[:4] / norm
    loss = m[0] + (BETA * m[1] if s["ref"] is not None else 0) - case["eta"] * m[2]
    return {"loss": loss, "stats": torch.cat([loss[None], m, norm[None]]), "logprobs": lps, "dlogits": out}


def _exact_balance(case, s):
    l = s["logits"].double().requires_grad_(True)
    T, E, k, B = case["T"], case["E"], case["k"], case["seqs"]
    ids = s["ids"].long()
    live = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    cuts = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    scores = torch.softmax(l, 1) if case["score"] == SOFTMAX else torch.sigmoid(l)
    q = scores / scores.sum(1, keepdim=True)
    counts = torch.zeros(B, E, dtype=torch.int32, device=DEV)
    bal, used = torch.zeros((), dtype=torch.float64, device=DEV), 0
    for b in range(B):
        on = torch.zeros(T, dtype=torch.bool, device=DEV)
        on[cuts[b]:cuts[b + 1]] = live[cuts[b]:cuts[b + 1]]
        m = int(on.sum())
        if not m:
            continue
        used += 1
        hits = torch.bincount(ids[on].reshape(-1), minlength=E)
        counts[b] = hits.int()
        bal = bal + (hits.double() * E / (k * m) * q[on].mean(0)).sum()
    bal = ALPHA * bal / max(used, 1)
    z = ZETA * (torch.logsumexp(l, 1)[live] ** 2).sum() / max(int(live.sum()), 1)
    total = bal + z
    if s["dg"] is not None:
        c = scores.gather(1, ids)
        total = total + (s["dg"].double() * ROUTE_SCALE * c / c.sum(1, keepdim=True)).sum()
    total.backward()
    return {"losses": torch.stack([bal, z]).detach(), "counts": counts, "d_logits": l.grad}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("logprobs", "policy"):
        return _exact_tokens(case, s)
    if case["op"] == "balance":
        return _exact_balance(case, s)
    wr, x = s["wr"].double(), s["x"].double()
    if case["op"] == "logits":
        return {"logits": torch.einsum("td,ed->te", x, wr)}
    dl = s["dl"].double()
    return {"dx": torch.einsum("te,ed->td", dl, wr), "dw": torch.einsum("te,td->ed", dl, x)}
