"""The training-step losses at the ends of their ranges.  The tolerances are
those of the operators' own tests, where they are derived."""
import pytest
import torch

pytestmark = pytest.mark.gpu
SIGMOID = 1


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
