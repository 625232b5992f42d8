"""The vocabulary losses (token log-probabilities, the clipped policy loss and
its gradient) against their 64-bit forms.

Tolerances.  One exponential carries the hardware's 2^-22 and its argument's
rounding, 2^-24 |z - max| twice (the scaled logit and the shift); a sum of V
terms adds at most ceil(V / 128) + 16 roundings of 2^-24 (128 lanes at the
least share a row, then a tree); so with R the row's range of finite z,
    rel = 2^-22 (8 + 2 min(R, 110)) + (V / 128 + 16) 2^-24
bounds p's relative and lp's absolute error (beyond 110 the exponential is
below fp32 altogether), beside lp's own rounding 2^-23 (|lp| + R).  A gradient
entry is a sum of parts, each a product of p and factors of lp: 4 rel of the
parts' absolute sum, 4 (|lp|'s error) of it through the ratio and exp(q); bf16
adds half a step, 2^-8."""
import math

import numpy as np
import pytest
import torch

from tests import loss_refs as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def _span(logits, tau, ok):
    z = logits.double() / tau
    fin = torch.isfinite(z)
    hi = torch.where(fin, z, -torch.inf).amax(1)
    lo = torch.where(fin & (z > hi[:, None] - 200), z, torch.inf).amin(1)
    return torch.where(ok & torch.isfinite(hi - lo), hi - lo, 0.0)


def _tol(logits, tau, lp, ok):
    V = logits.shape[1]
    span = _span(logits, tau, ok)
    rel = 2.0 ** -22 * (8 + 2 * span.clamp(max=110)) + (V / 128 + 16) * 2.0 ** -24
    at = rel + 2.0 ** -23 * (lp.abs().nan_to_num(0, 0, 0) + span)
    return rel, at


def _close(got, want, tol, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    same = (got == want) | torch.isnan(want)
    err = torch.where(same, 0.0, (got - want).abs())
    worst = (err / tol.clamp_min(2.0 ** -126)).max().item() if err.numel() else 0.0
    assert bool((err <= tol + 2.0 ** -126).all()), (what, worst)


def _rows(N, V, dt, seed, scale=3.0, ld=None, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = V if ld is None else ld
    flat = torch.full((off + N * ld + 8,), float("nan"), dtype=dt, device="cuda")
    x = flat[off:off + N * ld].view(N, ld)[:, :V] if N else flat[:0].view(0, V)
    if N:
        x.copy_(scale * torch.randn(N, V, device="cuda", generator=g))
    return x, g


def _inputs(N, V, g):
    y = torch.randint(0, V, (N,), device="cuda", generator=g)
    r = lambda: torch.randn(N, device="cuda", generator=g)  # noqa: E731
    return y, r()


def _check_logprobs(L, x, y, tau):
    lp, H = L.moe_token_logprobs(x, y, temperature=tau, entropy=True)
    want, wH, _, _, ok = R.token_rows(x, y.long(), tau)
    rel, at = _tol(x, tau, want, ok)
    _close(lp, want, at, "logprobs")
    # the entropy sums p |log p| with p's relative error and log p's absolute one
    _close(H, wH, (rel * (2 * wH + 4) + at).nan_to_num(0), "entropy")
    return lp, H


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,V,ld,off,tau", [
    (1, 1, None, 0, 1.0), (3, 2, None, 0, 1.0), (5, 7, 9, 1, 0.5), (2, 33, 40, 3, 1.0), (70, 1000, None, 0, 1.0),
    (4, 4097, 4099, 1, 1.3), (3, 32771, None, 0, 0.7), (600, 515, 520, 5, 1.0), (2, 131072, None, 0, 1.0),
    (1, 300001, None, 0, 1.0), (1300, 64, None, 0, 1.0), (9, 16384, 16385, 2, 1.0), (0, 64, None, 0, 1.0),
    (200, 20000, None, 0, 1.0), (37, 65536, None, 0, 2.0)])
def test_logprobs(L, dt, N, V, ld, off, tau):
    x, g = _rows(N, V, dt, 1000 * N + V, ld=ld, off=off)
    y, _ = _inputs(N, V, g)
    if N > 2:
        y[1] = -100
    _check_logprobs(L, x, y.int() if V % 2 else y, tau)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [64, 5000, 140000])
def test_logprobs_hard_rows(L, dt, V):
    """-inf and lowest-value masks, one logit left, all equal, huge, NaN, +inf, nothing left."""
    x, g = _rows(12, V, dt, V)
    y, _ = _inputs(12, V, g)
    ninf, low = float("-inf"), torch.finfo(dt).min
    x[0, V // 2:] = ninf
    y[0] = 3                                  # half of the row masked, target kept
    y[1] = V - 1
    x[1, V - 1] = ninf                        # the target itself masked
    x[2] = ninf
    x[2, 5] = 1.5
    y[2] = 5                                  # one logit left: lp = 0, H = 0
    x[3] = ninf                               # nothing left: not scored
    x[4] = low
    x[4, 1] = 0.0
    y[4] = 1
    x[5] = low                                # all at the lowest value: uniform
    x[6] = 0.25
    x[7, 3] = float("nan")
    x[8, 3] = float("inf")
    x[9] *= 300                               # exponentials far below fp32
    x[10] = float("nan")
    y[10] = -1                                # not scored whatever it holds
    x[11, :V - 1] = ninf
    y[11] = V - 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp, H = L.moe_token_logprobs(x, y, entropy=True, dev_status=st)
    assert int(st) == L.MOE_DEV_BAD_IDS                      # row 3
    want, wH, _, _, ok = R.token_rows(x, y, 1.0)
    assert not bool(ok[3]) and not bool(ok[10])
    rel, at = _tol(x, 1.0, want, ok)
    assert lp[1] == -torch.inf and torch.isnan(lp[7]) and torch.isnan(lp[8])
    assert lp[2] == 0 and H[2] == 0 and lp[3] == 0 and lp[10] == 0 and lp[11] == 0
    keep = torch.tensor([0, 2, 4, 5, 6, 9, 11], device="cuda")
    _close(lp[keep], want[keep], at[keep], "logprobs")
    _close(H[keep], wH[keep], (rel * (2 * wH + 4) + at)[keep], "entropy")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("tau,scale", [(1e-7, 1e-7), (1e5, 3e4), (1.0, 1e30), (3e-3, 0.02)])
def test_logprobs_extreme_scales(L, dt, tau, scale):
    """Temperatures and logits far from 1, a policy gradient among them."""
    x, g = _rows(6, 3001, dt, 77, scale=scale)
    y, _ = _inputs(6, 3001, g)
    lp, H = _check_logprobs(L, x, y, tau)
    assert torch.isfinite(H).all()
    old = lp.clamp(min=-50.0)
    _check_policy(L, x, y, old, torch.ones(6, device="cuda"), None, None, tau=tau, eta=0.01)


def test_logprobs_target_out_of_range(L):
    x, g = _rows(4, 100, F32, 1)
    y = torch.tensor([5, 100, -7, 2 ** 40], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lp, H = L.moe_token_logprobs(x, y, entropy=True, dev_status=st)
    assert int(st) == L.MOE_DEV_BAD_IDS
    assert lp[0] != 0 and lp[1:].eq(0).all() and H[1:].eq(0).all()
    st.zero_()
    L.moe_token_logprobs(x, y.clamp(max=99), dev_status=st)
    assert int(st) == 0


def _policy_case(N, V, dt, seed, tau=1.0, ld=None, off=0, prompt=0, scale=3.0):
    x, g = _rows(N, V, dt, seed, ld=ld, off=off, scale=scale)
    y, adv = _inputs(N, V, g)
    lp = R.token_rows(x, y, tau)[0]
    noise = 0.3 * torch.randn(N, device="cuda", generator=g).double()
    for b in (math.log(0.8), math.log(1.28)):
        noise = torch.where((noise - b).abs() < 1e-3, noise + 4e-3, noise)
    old = (lp - noise).float()
    ref = (lp + 0.2 * torch.randn(N, device="cuda", generator=g).double()).float()
    w = torch.rand(N, device="cuda", generator=g) + 0.25
    w[torch.arange(N, device="cuda") % 16 < prompt] = 0.0
    return x, y, old, adv, ref, w


def _check_policy(L, x, y, old, adv, ref, w, tau=1.0, beta=0.0, eta=0.0, norm=0.0, grad_scale=1.0, **kw):
    N, V = x.shape
    before = x.clone()
    stats, lp, d = L.moe_policy_loss(x, y, old, adv, ref_logprobs=ref, weights=w, temperature=tau, clip_low=0.2,
                                     clip_high=0.28, kl_coef=beta, entropy_coef=eta, norm=norm,
                                     grad_scale=grad_scale, **kw)
    want = R.policy(before, y.long(), old, adv, ref, w, tau, 0.2, 0.28, beta, eta, norm, grad_scale)
    ok = want["ok"]
    rel, at = _tol(before, tau, want["logprobs"], ok)
    _close(lp, want["logprobs"], at, "logprobs")
    if d is not None:
        # old and ref enter as given: lp - old has lp's error; exp() moves by that much relatively
        tol = want["size"] * (4 * rel + 4 * at + 2.0 ** -21)[:, None]
        if d.dtype == BF:
            tol = tol + 2.0 ** -8 * want["dlogits"].abs()
        _close(d, want["dlogits"], tol, "dlogits")
        assert d[~ok].eq(0).all()
    ws = torch.ones(N, dtype=torch.float64, device="cuda") if w is None else w.double()
    ws = torch.where(ok, ws, 0.0)
    nrm = float(want["stats"][5])
    err = float((ws * (4 * rel + 4 * at + 2.0 ** -20)).sum() / nrm) if nrm else 0.0
    big = float(torch.where(ok, adv.double().abs(), 0.0).max()) * 4 + 8 + math.log(V) if N else 1.0
    s = stats.double().cpu()
    assert float((s[:5] - want["stats"][:5]).abs().max()) <= err * big + 2.0 ** -23 * float(want["stats"][:5].abs().max()), \
        (s, want["stats"])
    assert abs(float(s[5]) - nrm) <= 2.0 ** -23 * abs(nrm)
    return stats, lp, d


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,V,ld,off,tau,beta,eta,prompt", [
    (1, 1, None, 0, 1.0, 0.1, 0.01, 0), (3, 2, None, 0, 1.0, 0.0, 0.0, 0), (5, 7, 9, 1, 0.5, 0.1, 0.02, 0),
    (64, 33, 40, 3, 1.0, 0.05, 0.0, 4), (70, 1000, None, 0, 1.0, 0.1, 0.0, 8), (4, 4097, 4099, 1, 1.3, 0.0, 0.01, 0),
    (33, 32771, None, 0, 0.7, 0.1, 0.01, 5), (700, 515, 520, 5, 1.0, 0.1, 0.0, 3), (2, 131072, None, 0, 1.0, 0.1, 0.0, 0),
    (1, 300001, None, 0, 1.0, 0.1, 0.0, 0), (1300, 64, None, 0, 1.0, 0.0, 0.01, 15), (160, 16384, None, 0, 1.0, 0.1, 0.0, 4),
    (310, 8200, None, 0, 1.0, 0.1, 0.01, 0), (40, 65536, 65544, 0, 1.0, 0.1, 0.0, 2)])
def test_policy(L, dt, N, V, ld, off, tau, beta, eta, prompt):
    x, y, old, adv, ref, w = _policy_case(N, V, dt, N + V, tau, ld, off, prompt)
    _check_policy(L, x, y, old, adv, ref if beta else None, w, tau, beta, eta)


def test_policy_arguments(L):
    """No weights, a given norm, a loss scale, no gradient, int32 targets, the gradient with a row stride."""
    x, y, old, adv, ref, w = _policy_case(50, 1003, F32, 3)
    _check_policy(L, x, y.int(), old, adv, ref, None, beta=0.1, norm=17.0, grad_scale=4.0)
    s, lp, d = _check_policy(L, x, y, old, adv, None, w, dlogits=False)
    assert d is None
    wide = torch.full((50, 1100), 7.0, device="cuda")
    _check_policy(L, x, y, old, adv, ref, w, beta=0.1, dlogits=wide[:, 3:1006])
    assert wide[:, :3].eq(7).all() and wide[:, 1006:].eq(7).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,V", [(40, 4096), (3, 150000), (400, 1001)])
def test_policy_gradient_over_the_logits(L, dt, N, V):
    """dlogits written over the logits: the same bits as apart."""
    x, y, old, adv, ref, w = _policy_case(N, V, dt, 5, prompt=3)
    kw = dict(ref_logprobs=ref, weights=w, kl_coef=0.1, entropy_coef=0.01)
    s0, l0, d0 = L.moe_policy_loss(x, y, old, adv, **kw)
    z = x.clone()
    s1, l1, d1 = L.moe_policy_loss(z, y, old, adv, dlogits=z, **kw)
    assert d1.data_ptr() == z.data_ptr()
    assert torch.equal(d0, d1) and torch.equal(s0, s1) and torch.equal(l0, l1)
    s2, l2, d2 = L.moe_policy_loss(x, y, old, adv, **kw)                       # and the same bits again
    assert torch.equal(d0, d2) and torch.equal(s0, s2) and torch.equal(l0, l2)


@pytest.mark.parametrize("dt", [BF, F32])
def test_policy_masked_rows_hold_anything(L, dt):
    x, y, old, adv, ref, w = _policy_case(64, 777, dt, 9, prompt=6)
    off = w == 0
    bad = [x.clone(), y.clone(), old.clone(), adv.clone(), ref.clone(), w]
    for t in (bad[0], bad[2], bad[3], bad[4]):
        t[off] = float("nan")
    bad[1][off] = 2 ** 50
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = _check_policy(L, x, y, old, adv, ref, w, beta=0.1, eta=0.01)
    b = L.moe_policy_loss(bad[0], bad[1], bad[2], bad[3], ref_logprobs=bad[4], weights=w, clip_high=0.28,
                          kl_coef=0.1, entropy_coef=0.01, dev_status=st)
    assert int(st) == 0
    for u, v in zip(a, b):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dt", [BF, F32])
def test_policy_hard_rows(L, dt):
    V = 3000
    x, y, old, adv, ref, w = _policy_case(10, V, dt, 4)
    ninf = float("-inf")
    x[0, 7:] = ninf
    y[0] = 2
    x[1, 5] = ninf
    y[1] = 5                       # the target masked: ratio 0, log p = -inf
    adv[1] = 1.0
    x[2] = ninf                    # nothing left: not scored
    adv[3] = 0.0
    old[3] = -1000.0               # a ratio beyond fp32 with advantage 0
    adv[4] = 1.0
    old[4] = -1000.0               # ... clipped with a positive one
    x[5] = torch.finfo(dt).min
    x[5, 9] = 1.0
    y[5] = 9
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = L.moe_policy_loss(x, y, old, adv, weights=w, entropy_coef=0.01, dev_status=st)
    assert int(st) == L.MOE_DEV_BAD_IDS
    want = R.policy(x, y, old, adv, None, w, 1.0, 0.2, 0.2, 0.0, 0.01)
    assert not want["ok"][2] and got[2][2].eq(0).all() and got[1][2] == 0
    assert got[1][1] == ninf
    rel, at = _tol(x, 1.0, want["logprobs"], want["ok"])
    tol = want["size"] * (4 * rel + 4 * at + 2.0 ** -21)[:, None] + (2.0 ** -8 if dt == BF else 0) * want["dlogits"].abs()
    _close(got[2], want["dlogits"], tol, "dlogits")
    assert torch.isfinite(got[0]).all()
    # all weights 0: zeros, no division by the empty sum
    s, lp, d = L.moe_policy_loss(x, y, old, adv, weights=torch.zeros_like(w))
    assert s.eq(0).all() and d.eq(0).all() and lp.eq(0).all()


def test_policy_empty(L):
    e = torch.empty(0, device="cuda")
    s, lp, d = L.moe_policy_loss(torch.empty(0, 40, device="cuda"), e.long(), e, e)
    assert s.eq(0).all() and lp.numel() == 0 and d.shape == (0, 40)


def test_policy_gradient_against_differences(L):
    """Central differences of the 64-bit loss: with step h the difference is off
    by the third derivative, < h^2 of the entries' scale (h = 1e-4: 1e-8)."""
    x, y, old, adv, ref, w = _policy_case(6, 50, F32, 12, tau=0.9)
    kw = dict(tau=0.9, lo=0.2, hi=0.28, beta=0.1, eta=0.05)
    _, _, d = L.moe_policy_loss(x, y, old, adv, ref_logprobs=ref, weights=w, temperature=0.9, clip_low=0.2,
                                clip_high=0.28, kl_coef=0.1, entropy_coef=0.05)
    h = 1e-4
    xd = x.double()
    for t, v in [(0, 3), (1, int(y[1])), (2, 49), (3, int(y[3])), (5, 0)]:
        up, dn = xd.clone(), xd.clone()
        up[t, v] += h
        dn[t, v] -= h
        f = lambda z: float(R.policy(z, y, old, adv, ref, w, **kw)["stats"][0])  # noqa: E731
        num = (f(up) - f(dn)) / (2 * h)
        assert abs(num - float(d[t, v])) < 1e-6 * max(1.0, abs(num)), (t, v, num, float(d[t, v]))


def test_losses_follow_the_stream_and_graphs(L):
    """Inputs made and used on another stream; the calls captured and replayed on new inputs."""
    x, y, old, adv, ref, w = _policy_case(48, 5000, BF, 21, prompt=2)
    kw = dict(ref_logprobs=ref, weights=w, kl_coef=0.1)
    want = L.moe_policy_loss(x, y, old, adv, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(L.moe_policy_loss_workspace_size(48, 5000), dtype=torch.uint8, device="cuda")
    with torch.cuda.stream(side):
        z = x * 1.0
        got = L.moe_policy_loss(z, y, old, adv, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    z = torch.zeros_like(x)
    st, lp, dl = torch.empty(6, device="cuda"), torch.empty(48, device="cuda"), torch.empty_like(x)
    lp2, H = torch.empty(48, device="cuda"), torch.empty(48, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.moe_policy_loss(z, y, old, adv, stats=st, logprobs=lp, dlogits=dl, workspace=ws, **kw)
        L.moe_token_logprobs(z, y, logprobs=lp2, entropy=H)
    for _ in range(2):
        z.copy_(x)
        dl.fill_(3)
        g.replay()
        assert torch.equal(want[0], st) and torch.equal(want[1], lp) and torch.equal(want[2], dl)
    ones = L.moe_token_logprobs(x, y)[0]
    assert torch.equal(torch.where(w != 0, lp2, 0.0), torch.where(w != 0, ones, 0.0))


@pytest.mark.parametrize("V", [4096, 140000])
def test_rows_beyond_32_bit_offsets(L, V):
    """Row starts beyond 2^32 elements (a row stride of 2^31 + 24)."""
    ld, N = 2 ** 31 + 24, 3
    flat = torch.empty((N - 1) * ld + V, dtype=BF, device="cuda")
    x = flat.as_strided((N, V), (ld, 1))
    src, y, old, adv, ref, w = _policy_case(N, V, BF, 8)
    x.copy_(src)
    a = L.moe_policy_loss(src, y, old, adv, weights=w)
    b = L.moe_policy_loss(x, y, old, adv, weights=w)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    assert torch.equal(L.moe_token_logprobs(src, y)[0], L.moe_token_logprobs(x, y)[0])
    L.moe_policy_loss(x, y, old, adv, weights=w, dlogits=x)
    assert torch.equal(x, a[2])


@pytest.mark.parametrize("N", [1, 33, 511, 512, 513, 2100])
def test_policy_norm_at_every_row_count(L, N):
    """The weights' sum as the norm, by the rows or before them: the stats and
    the gradient equal those of the call that is given it; a negative sum and
    one of zero hold too."""
    x, y, old, adv, ref, w = _policy_case(N, 100, F32, 70 + N)
    for v in (w, -w, torch.zeros_like(w)):
        norm = v.double().sum()
        st, lp, dl = L.moe_policy_loss(x, y, old, adv, ref_logprobs=ref, weights=v, kl_coef=0.1, entropy_coef=0.02)
        assert abs(st[5].double() - norm) <= 2.0 ** -23 * abs(norm)
        if v is w:
            st1, lp1, dl1 = L.moe_policy_loss(x, y, old, adv, ref_logprobs=ref, weights=v, kl_coef=0.1,
                                              entropy_coef=0.02, norm=float(st[5]))
            assert torch.equal(st, st1) and torch.equal(lp, lp1)
            keep = st, dl
            # norms one step apart and five roundings after them, 6 * 2^-23;
            # the target's entry cancels, so 2^-18 of the largest
            assert (dl - dl1).abs().max() <= 2.0 ** -18 * dl.abs().max()
        elif v.any():
            # numerators and norm change their signs together
            assert torch.equal(st[:5], keep[0][:5]) and (dl - keep[1]).abs().max() <= 2.0 ** -18 * dl.abs().max()
        else:
            assert st.eq(0).all() and dl.eq(0).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("v", [1, 2, 4, 5, 7, 9, 11, 13, 15, 17, 19, 25])
def test_rows_of_every_chunk(L, dt, v):
    """v vectors of 16 bytes a thread of 128 (log-probabilities) or 256
    (gradients), the last one short, rows on odd starts and on vectors."""
    W = 8 if dt == BF else 4
    N = 320
    for V, ld, off in ((128 * W * v - W - 1, None, 3), (128 * W * v, None, 0)):
        x, g = _rows(N, V, dt, v, ld=ld, off=off)
        y, _ = _inputs(N, V, g)
        y[::7] = V - 1
        y[1::7] = 0
        _check_logprobs(L, x, y, 1.1)
    for V, off, eta in ((256 * W * v - W - 1, 3, 0.01), (256 * W * v, 0, 0.0)):
        x, y, old, adv, ref, w = _policy_case(N, V, dt, v, 1.0, None, off, 1)
        _check_policy(L, x, y, old, adv, ref, w, 1.0, 0.1, eta)
