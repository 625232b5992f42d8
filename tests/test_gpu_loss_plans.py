"""Every way the vocabulary losses spread a row (threads of a CTA, CTAs of a
cluster, vectors a thread, in registers or through the ring), and the one-CTA
count of the balance loss.  The choice of spread is restated here so that the
test knows which kernels its sizes reach; tolerances as in the operators' own
tests."""
import pytest
import torch

from tests import loss_refs as R
from tests import test_gpu_losses as TL

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def _plan(N, V, w, aligned, policy, sms):
    """(threads of the kernel, vectors a thread, ring, CTAs)."""
    nvec = -(-V // w) + (not aligned)
    fill, C, threads = 4 * sms, 2 if policy and nvec > 8192 else 1, 32
    most = 256 if (policy and nvec > 2048) or 8 * N <= fill else 128
    while threads < most and threads * 8 < nvec:
        threads *= 2
    while C < 8 and N * C * 2 <= fill and C * threads < nvec:
        C *= 2
    v = -(-nvec // (C * threads))
    chunks = -(-v // 8)
    ring, NV = policy and chunks > 1, -(-v // chunks)
    NV = 4 if NV == 3 else NV
    if NV > 4 and (not ring if policy else threads > 128):
        NV += NV % 2
    return 256 if threads > 128 else 128, NV, ring, C


# rows and vectors of 16 bytes: few rows on wide CTAs and clusters, many on narrow ones
SIZES = [(N, v) for N in (1, 20, 64) for v in (40, 200, 1100, 2100, 5000, 9000, 13000)] + \
    [(400, v) for v in (30, 60, 100, 600, 700, 800, 1000, 1100, 1300, 1500, 1700, 1800, 2000, 2100, 2500, 3000, 3300, 3500, 4000)] + \
    [(2, 15000), (5, 33000), (90, 1030), (90, 1500), (90, 1700), (90, 2000), (160, 2300), (160, 2800), (160, 3500), (160, 4000),
     (160, 9000)]


def _reached(policy, sms):
    return {_plan(N, v * 8 - 3, 8, False, policy, sms)[:3] for N, v in SIZES} | \
        {_plan(N, v * 8, 8, True, policy, sms)[:3] for N, v in SIZES}


def test_sizes_reach_every_kernel(L):
    sms = L.moe_device_sm_count()
    lp = {(256, n, False) for n in (1, 2, 4, 6, 8)} | {(128, n, False) for n in (1, 2, 4, 5, 6, 7, 8)}
    po = {(t, n, False) for t in (128, 256) for n in (1, 2, 4, 6, 8)} | {(t, n, True) for t in (128, 256) for n in (5, 6, 7, 8)}
    assert _reached(False, sms) == lp, lp ^ _reached(False, sms)
    assert _reached(True, sms) == po, po ^ _reached(True, sms)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,v", SIZES)
def test_every_spread(L, dt, N, v):
    """Whole vectors on an aligned start, and a row that is short of its last
    vector on an odd one; with an entropy bonus and without."""
    W = 8 if dt == BF else 4
    for V, off, eta in ((v * W, 0, 0.0), (v * W - 3, 1, 0.01)):
        x, y, old, adv, ref, w = TL._policy_case(N, V, dt, N + V, 1.0, None, off, 1 if N > 1 else 0)
        TL._check_policy(L, x, y, old, adv, ref, w, 1.0, 0.1, eta)
        y[::3] = V - 1
        y[1::3] = 0
        TL._check_logprobs(L, x, y, 1.0)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (37, 8, 2), (200, 64, 6), (256, 33, 8), (128, 200, 5), (60, 1000, 32)])
def test_balance_counted_by_one_cta(L, score, T, E, k):
    """Few tokens and no offsets: masked tokens and ids out of range are not counted."""
    g = torch.Generator(device="cuda").manual_seed(T)
    l = 2 * torch.randn(T, E, device="cuda", generator=g)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int()
    m = torch.rand(T, device="cuda", generator=g) < 0.6
    m[0] = True
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    losses, counts, d = L.moe_balance_loss(l, ids, score, 0.1, z_coef=0.01, token_mask=m, dev_status=st)
    wl, wc, wd = R.balance(l, ids, score, 0.1, 0.01, m)
    assert int(st) == 0 and torch.equal(counts.long(), wc)
    # the balance tests' relative bound, on the losses and on the norm of the gradient
    span = float((l.amax(1) - l.amin(1)).max())
    rel = 2.0 ** -24 * (24 + 2 * min(span, 110) + E / 16)
    assert bool(((losses.double() - wl).abs() <= 4 * rel * wl.abs() + 1e-30).all())
    assert d[~m].eq(0).all()
    # entries are differences f - sum f q: the bound is on their parts, q (f + sum f q) and 2 lse p
    q = torch.softmax(l.double(), 1) if score == 0 else torch.sigmoid(l.double()) / torch.sigmoid(l.double()).sum(1, keepdim=True)
    n = int(m.sum())
    f = wc[0].double() * E / (k * n)
    size = 0.1 / n * q * (f + (q * f).sum(1, keepdim=True)) + \
        0.02 / n * (torch.logsumexp(l.double(), 1, keepdim=True).abs() + 1) * torch.softmax(l.double(), 1)
    assert bool(((d.double() - wd).abs() <= 4 * rel * size + 1e-35).all())
    if T > 30:
        at = int(torch.nonzero(m)[3])
        bad = ids.clone()
        bad[at, 0], bad[at, k - 1] = -1, E
        losses, counts, _ = L.moe_balance_loss(l, bad, score, 0.1, token_mask=m, dev_status=st)
        assert int(st) == L.MOE_DEV_BAD_IDS and int(counts.sum()) == n * k - 2
        want = wc[0].clone()
        want[ids[at, 0].long()] -= 1
        want[ids[at, k - 1].long()] -= 1
        assert torch.equal(counts[0].long(), want)
