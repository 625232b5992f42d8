"""The training-step losses at the ends of their ranges.  The tolerances are
those of the operators' own tests, where they are derived."""
import pytest
import torch

from tests import loss_refs as R

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = 0, 1


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


# ------------------------------------------------------------ balance loss

def _check_sigmoid(L, l, ids, alpha=0.1, zeta=0.0):
    """One sequence, sigmoid scores, from log sigmoid: q = softmax(log sigmoid(l))
    holds where sigmoid itself underflows in 64 bits."""
    T, E = l.shape
    k = ids.shape[1]
    losses, counts, d = L.moe_balance_loss(l, ids, SIGMOID, alpha, z_coef=zeta)
    z = l.double().requires_grad_(True)
    q = torch.softmax(torch.nn.functional.logsigmoid(z), 1)
    n = torch.bincount(ids.long().reshape(-1), minlength=E).double()
    lse = torch.logsumexp(z, 1)
    want = torch.stack([alpha * (n * E / (k * T) * q.mean(0)).sum(), zeta * (lse ** 2).mean()])
    (wd,) = torch.autograd.grad(want.sum(), z)
    want, q, lse = want.detach(), q.detach(), lse.detach()
    assert torch.equal(counts[0].double(), n)
    span = float((l.double().amax(1) - l.double().amin(1)).max())
    rel = 2.0 ** -24 * (24 + 2 * min(span, 110) + E / 16)
    assert bool(((losses.double() - want).abs() <= 4 * rel * want.abs() + 1e-30).all()), (losses, want)
    size = 2 * alpha * float(n.max()) * E / (k * T) / T * q + \
        2 * zeta * (lse.abs() + 1)[:, None] / T * torch.softmax(l.double(), 1)
    err = (d.double() - wd).abs()
    assert bool((err <= 4 * rel * size + 1e-35).all()), float((err / size).nan_to_num(1e30).max() / rel)


@pytest.mark.parametrize("E", [8, 40, 100, 256, 512, 1000])
@pytest.mark.parametrize("base", [-5.0, -30.0, -48.0, -52.0, -60.0, -87.0, -100.0, -3000.0, -1e9])
@pytest.mark.parametrize("mixed", [False, True])
def test_balance_sigmoid_low_tokens(L, E, base, mixed):
    """Tokens whose logits are all low, alone and among ordinary ones: q and its
    slope stay those of 64 bits, down to a mask of -1e9 (q uniform there)."""
    T, k = 203, 4
    g = torch.Generator(device="cuda").manual_seed(E)
    l = torch.randn(T, E, device="cuda", generator=g)
    low = torch.arange(T, device="cuda") % 3 > 0 if mixed else torch.ones(T, dtype=torch.bool, device="cuda")
    l[low] += base
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int()
    _check_sigmoid(L, l, ids)
    _check_sigmoid(L, l, ids, zeta=0.01)


def test_balance_sigmoid_low_experts(L):
    """Experts at -40 to -86 below one at 1: slopes s (1 - s) where s s underflows."""
    T, E = 200, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    l = -40 - 46 * torch.rand(T, E, device="cuda", generator=g)
    l[:, 5] = 1.0
    ids = torch.rand(T, E, device="cuda", generator=g).topk(3, 1).indices.int()
    _check_sigmoid(L, l, ids)


@pytest.mark.parametrize("E,k", [(8, 2), (64, 6), (256, 8), (300, 1), (1000, 32)])
@pytest.mark.parametrize("base", [-40.0, -80.0, -84.0, -87.0, -88.0, -95.0, -1000.0, -1e9])
@pytest.mark.parametrize("mixed", [False, True])
def test_gates_gradient_of_low_tokens(L, E, k, base, mixed):
    """Renormalised sigmoid gates of tokens whose logits are all low: from log
    sigmoid, as their ratios are; plain ones have a derivative below fp32."""
    T = 203
    g = torch.Generator(device="cuda").manual_seed(E + k)
    l = torch.randn(T, E, device="cuda", generator=g)
    low = torch.arange(T, device="cuda") % 3 > 0 if mixed else torch.ones(T, dtype=torch.bool, device="cuda")
    l[low] += base
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices
    dg = 1e-2 * torch.randn(T, k, device="cuda", generator=g)
    z = l.double().gather(1, ids)
    p = torch.softmax(torch.nn.functional.logsigmoid(z), 1)
    want = 1.5 * p * torch.sigmoid(-z) * (dg.double() - (p * dg.double()).sum(1, keepdim=True))
    d = L.moe_balance_loss(l, ids.int(), SIGMOID, 0.0, d_gates=dg, route_scale=1.5)[2]
    rel = 2.0 ** -24 * (24 + 2 * min(float((l.amax(1) - l.amin(1)).max()), 110) + E / 16)
    size = 2 * 1.5 * dg.double().abs().sum(1, keepdim=True)
    assert bool(((d.gather(1, ids).double() - want).abs() <= 4 * rel * size).all())
    assert d.scatter(1, ids, 0.0).eq(0).all()
    d = L.moe_balance_loss(l, ids.int(), SIGMOID, 0.0, d_gates=dg, renorm=0)[2]
    want = torch.sigmoid(z) * torch.sigmoid(-z) * dg.double()
    assert bool(((d.gather(1, ids).double() - want).abs() <= 4 * rel * want.abs() + 1e-35).all())


def test_balance_sums_beyond_fp32(L):
    """A z loss beyond fp32 is an infinity; the balance loss beside it stays."""
    for T in (40, 3000):
        g = torch.Generator(device="cuda").manual_seed(2)
        l = torch.randn(T, 64, device="cuda", generator=g)
        l[3, 4] = l[9, 1] = 1e30
        ids = torch.rand(T, 64, device="cuda", generator=g).topk(2, 1).indices.int()
        losses, _, d = L.moe_balance_loss(l, ids, SOFTMAX, 0.1, z_coef=1e-4)
        want = R.balance(l, ids, SOFTMAX, 0.1)[0]
        assert losses[1] == torch.inf and not d.isnan().any()
        assert abs(float(losses[0]) - float(want[0])) <= 2.0 ** -18 * float(want[0])


# ---------------------------------------------------------- dense backward

@pytest.mark.parametrize("T,d,E", [(200, 256, 64), (333, 384, 37), (1500, 512, 256), (4000, 7168, 256)])
def test_router_backward_dense_infinite_operands(L, T, d, E):
    """Infinities and NaN in x and W_r give what the products of fp32 give, also
    against gradients of few bits (a part of theirs that is 0 times an infinity
    is no NaN) and exact zeros (where it is one)."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    inf, nan = float("inf"), float("nan")
    dl = torch.randn(T, E, device="cuda", generator=g)
    dl[:, ::2] = dl[:, ::2].bfloat16().float()
    dl[10:20] = 1.0
    dl[20:25] = -0.5
    dl[26] = 2.0 ** -100
    dl[27] = -2.0 ** -126
    dl[::7, 2] = 0.0
    dl[40, 6] = inf
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    w = (0.05 * torch.randn(E, d, device="cuda", generator=g)).bfloat16()
    x[12, 5], x[22, 9], x[26, 70], x[27, 71], x[30, 3], x[7, 100], x[40, 101] = inf, -inf, inf, inf, nan, inf, -inf
    x[10, 200], x[21, 200] = inf, inf
    w[2, 4], w[6, 8], w[2, 10], w[7, 10], w[8, 20] = inf, -inf, inf, inf, nan
    dx, dw = L.moe_router_backward_dense(x, w, dl)
    for got, a, b in ((dx, dl.double(), w.double()), (dw, dl.double().t(), x.double())):
        want = a @ b
        assert not want.isfinite().all()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got == inf, want == inf) and torch.equal(got == -inf, want == -inf)
        fin = want.isfinite()
        bound = (a.shape[1] + 64) * 2.0 ** -24 * (a.abs() @ b.abs()) + 2.0 ** -126
        assert bool(((got.double() - want).abs()[fin] <= bound[fin]).all())


# --------------------------------------------------------- vocabulary rows

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tau", [1e20, 1e27, 1e30, 3e38])
@pytest.mark.parametrize("V", [64, 5000])
def test_masked_logits_at_high_temperatures(L, dt, tau, V):
    """A logit of -inf has probability 0 whatever the temperature: the others
    are uniform."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (3 * torch.randn(6, V, device="cuda", generator=g)).to(dt)
    x[:, 1::3] = float("-inf")
    y = torch.tensor([0, 2, 3, 5, 6, 8], device="cuda")
    lp, H = L.moe_token_logprobs(x, y, temperature=tau, entropy=True)
    want, wH, _, _, _ = R.token_rows(x, y, tau)
    # the rows' bound with a range of 0: 2^-22 8 + (V / 128 + 16) 2^-24 and lp's own roundings
    rel = 2.0 ** -22 * 8 + (V / 128 + 16) * 2.0 ** -24
    assert bool(((lp.double() - want).abs() <= rel + 2.0 ** -23 * want.abs()).all())
    assert bool(((H.double() - wH).abs() <= rel * (2 * wH + 5) + 2.0 ** -23 * wH).all())
    d = L.moe_policy_loss(x, y, lp, torch.ones(6, device="cuda"), temperature=tau, grad_scale=1e30)[2]
    assert d[:, 1::3].eq(0).all() and d.isfinite().all()


@pytest.mark.parametrize("N", [40, 1100])
def test_policy_sums_beyond_fp32(L, N):
    """A policy term that sums beyond fp32 is an infinity, not a NaN; the other means stay."""
    g = torch.Generator(device="cuda").manual_seed(N)
    x = torch.randn(N, 100, device="cuda", generator=g)
    y = torch.randint(0, 100, (N,), device="cuda", generator=g)
    lp, H = L.moe_token_logprobs(x, y, entropy=True)
    adv = torch.full((N,), 1e38, device="cuda")
    for s in (1, -1):
        st = L.moe_policy_loss(x, y, lp, s * adv, weights=torch.ones(N, device="cuda"))[0]
        assert st[0] == -s * torch.inf and st[1] == -s * torch.inf
        assert st[2] == 0 and st[4] == 0 and st[5] == N
        # a KL mean beyond fp32 stays out of the loss where its coefficient is 0
        st2 = L.moe_policy_loss(x, y, lp, s * torch.ones(N, device="cuda"), ref_logprobs=lp + 100,
                                weights=torch.full((N,), 1e4, device="cuda"))[0]
        assert st2[2] == torch.inf and abs(float(st2[0]) + s) <= 2.0 ** -20
        # N entropies summed in two fp32 numbers, one division, against their own fp32 values
        assert abs(float(st[3]) - float(H.double().mean())) <= 2.0 ** -22 * float(H.double().mean())
