"""Plain 64-bit forms of the training-step losses, from their definitions, for
the tests (torch double, any device; no code of the package)."""
import torch


def token_rows(logits, targets, tau, scored=None):
    """(logprob, entropy, log p, p, scored) in 64 bits; unscored rows 0."""
    V = logits.shape[1]
    z = logits.double() / tau
    ok = (targets >= 0) & (targets < V) & ~(z == -torch.inf).all(1)
    if scored is not None:
        ok = ok & scored
    z = torch.where(ok[:, None], z, 0.0)
    z = z - z.amax(1, keepdim=True)         # first: a row at the type's lowest value swallows its log-sum otherwise
    logp = z - torch.logsumexp(z, 1, keepdim=True)
    p = logp.exp()
    H = -torch.where(p > 0, p * logp, torch.where(p.isnan(), p, 0.0)).sum(1)
    lp = logp.gather(1, targets.long().clamp(0, V - 1)[:, None])[:, 0]
    return torch.where(ok, lp, 0.0), torch.where(ok, H, 0.0), logp, p, ok


def policy(logits, targets, old, adv, ref=None, w=None, tau=1.0, lo=0.2, hi=0.2, beta=0.0, eta=0.0, norm=0.0,
           grad_scale=1.0):
    """dict of stats [6], logprobs, dlogits and `size` (the sum of the absolute
    parts of each gradient entry) in 64 bits."""
    N, V = logits.shape
    w = torch.ones(N, dtype=torch.float64, device=logits.device) if w is None else w.double()
    lp, H, logp, p, ok = token_rows(logits, targets, tau, w != 0)
    z = lambda v: torch.where(ok, v.double(), 0.0)  # noqa: E731
    A, old, wl = z(adv), z(old), z(w)
    r = torch.exp((lp - old).clamp(max=80.0))
    p0, p1 = -A * r, -A * r.clamp(1 - lo, 1 + hi)
    off = (p1 > p0) & ok
    g = torch.where(off, 0.0, p0)
    kl = torch.zeros_like(lp)
    gsize = g.abs()
    if ref is not None:
        q = (z(ref) - lp).clamp(max=80.0)
        kl = torch.where(ok, torch.expm1(q) - q, 0.0)
        g = g - beta * torch.expm1(q)
        gsize = gsize + abs(beta) * (torch.exp(q) + 1)
    nrm = norm if norm > 0 else float(w.sum())
    inv = 1.0 / nrm if nrm != 0 else 0.0
    m = [float((wl * torch.where(ok, v.double(), 0.0)).sum()) * inv for v in (torch.maximum(p0, p1), kl, H, off)]
    stats = torch.tensor([m[0] + (beta if ref is not None else 0.0) * m[1] - eta * m[2], *m, nrm],
                         dtype=torch.float64)
    coef = (grad_scale * inv / tau * wl)[:, None]
    lq = torch.where(p > 0, logp, torch.where(p.isnan(), p, 0.0))
    d = -g[:, None] * p + eta * p * (lq + H[:, None])
    size = gsize[:, None] * p + abs(eta) * p * (lq.abs() + H[:, None])
    at = targets.long().clamp(0, V - 1)[:, None]
    d = d.scatter_add(1, at, g[:, None])
    size = size.scatter_add(1, at, gsize[:, None])
    keep = ok[:, None]
    return dict(stats=stats, logprobs=lp, dlogits=torch.where(keep, coef * d, 0.0),
                size=torch.where(keep, coef.abs() * size, 0.0), ok=ok)


def gates(logits, ids, score_fn, renorm, scale):
    s = torch.softmax(logits, 1) if score_fn == 0 else torch.sigmoid(logits)
    c = s.gather(1, ids)
    return scale * (c / c.sum(1, keepdim=True) if renorm else c)


def balance(logits, ids, score_fn, alpha, zeta=0.0, mask=None, offsets=None, d_gates=None, renorm=1, scale=1.0,
            grad_scale=1.0):
    """(losses [2], counts [B, E], d_logits) in 64 bits; the gradient by
    autograd.  Ids in [0, E), distinct; offsets increasing."""
    T, E = logits.shape
    k = ids.shape[1]
    l = logits.double().clone().requires_grad_(True)
    cuts = [0, T] if offsets is None else [int(v) for v in offsets]
    live = torch.ones(T, dtype=torch.bool, device=logits.device) if mask is None else mask.bool()
    B = len(cuts) - 1
    counts = torch.zeros(B, E, dtype=torch.int64, device=logits.device)
    bal = torch.zeros((), dtype=torch.float64, device=logits.device)
    zsum, n, used = bal, 0, 0
    for b in range(B):
        on = torch.zeros(T, dtype=torch.bool, device=logits.device)
        on[cuts[b]:cuts[b + 1]] = live[cuts[b]:cuts[b + 1]]
        m = int(on.sum())
        if m == 0:
            continue
        used, n = used + 1, n + m
        counts[b] = torch.bincount(ids.long()[on].reshape(-1), minlength=E)
        fin = on & ~(l.detach() == -torch.inf).all(1)
        s = torch.softmax(l[fin], 1) if score_fn == 0 else torch.sigmoid(l[fin])
        q = s / s.sum(1, keepdim=True)
        f = counts[b].double() * E / (k * m)
        bal = bal + (f * q.sum(0) / m).sum()
        zsum = zsum + (torch.logsumexp(l[fin], 1) ** 2).sum()
    losses = torch.stack([alpha * bal / max(used, 1), zeta * zsum / max(n, 1)])
    total = grad_scale * losses.sum()
    if d_gates is not None:
        total = total + (gates(l, ids.long(), score_fn, renorm, scale) * d_gates.double()).sum()
    d = torch.zeros_like(l)
    if total.requires_grad:
        (d,) = torch.autograd.grad(total, l)
    return losses.detach(), counts, d
