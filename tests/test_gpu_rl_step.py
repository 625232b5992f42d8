"""The losses as a training step uses them: the layer's router_losses against
64-bit forms, and the example's step end to end."""
import pytest
import torch

from tests import loss_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def _layer(E, k, score_fn, renorm, T_max=512, d=256, F=128, seed=0):
    from block_scaled_fp8_router_gb300.layer import MoELayerFP8, MoEWeightsFP8, quantize_weights
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = MoEWeightsFP8((0.1 * r(E, d)).bfloat16(), *quantize_weights((0.06 * r(E, 2 * F, d)).bfloat16(),
                                                                    (0.06 * r(E, d, F)).bfloat16()))
    return MoELayerFP8(w, T_max, k, score_fn, renorm=renorm, route_scale=1.5), g


@pytest.mark.parametrize("score,renorm,replay,T", [(0, 0, False, 300), (0, 1, True, 512), (1, 1, True, 37), (1, 0, False, 129)])
def test_layer_router_losses(L, score, renorm, replay, T):
    """Products of the 64-bit gradient: d_logits within 2^-18 of its rows' size
    (the balance bound at E = 40) and the products' roundings beside it."""
    if replay and score == 0 and renorm == 0:
        pytest.skip("not replayed")
    E, k = 40, 3
    layer, g = _layer(E, k, score, renorm)
    x = torch.randn(T, 256, device="cuda", generator=g).bfloat16()
    rep = None
    if replay:
        rep = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int().t().contiguous()
    layer.forward(x, replay_kT=rep, train=True)
    dg = 1e-2 * torch.randn(T, k, device="cuda", generator=g)
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    mask = torch.rand(T, device="cuda", generator=g) < 0.8
    losses, counts, dx, dw = layer.router_losses(0.1, 0.01, d_gates=dg, token_mask=mask, seq_offsets=off, grad_scale=2.0)
    assert L.check_status(layer.dev_status) == 0
    ids = layer.ids[:T]
    if replay:
        assert torch.equal(ids, rep.t())
    l = x.double() @ layer.w.w_router.double().t()
    wl, wc, wd = R.balance(l, ids, score, 0.1, 0.01, mask, off, dg, renorm, 1.5, 2.0)
    assert torch.equal(counts.long(), wc)
    assert bool(((losses.double() - wl).abs() <= 2.0 ** -18 * wl).all())
    row = wd.abs().sum(1, keepdim=True)
    wdx, sdx = wd @ layer.w.w_router.double(), row * layer.w.w_router.double().abs().amax(0)
    assert bool(((dx.double() - wdx).abs() <= 2.0 ** -16 * sdx + 1e-12).all())
    wdw, sdw = wd.t() @ x.double(), row.t() @ x.double().abs()
    assert bool(((dw.double() - wdw).abs() <= 2.0 ** -16 * sdw + 1e-12).all())
    a = layer.router_losses(0.1, 0.01, d_gates=dg, token_mask=mask, seq_offsets=off, grad_scale=2.0)
    for u, v in zip((losses, counts, dx, dw), a):
        assert torch.equal(u, v)


def test_router_losses_agree_with_the_chosen_logits_backward(L):
    """With both coefficients 0 only the gates remain: router_backward's sums."""
    layer, g = _layer(32, 4, 1, 1)
    x = torch.randn(200, 256, device="cuda", generator=g).bfloat16()
    layer.forward(x, train=True)
    dg = torch.randn(200, 4, device="cuda", generator=g)
    dx0, dw0 = (t.clone() for t in layer.router_backward(dg))
    losses, counts, dx, dw = layer.router_losses(0.0, 0.0, d_gates=dg)
    assert losses.eq(0).all() and torch.equal(counts[0], layer.counts)
    assert float((dx - dx0).norm()) <= 2.0 ** -18 * float(dx0.norm())
    assert float((dw - dw0).norm()) <= 2.0 ** -18 * float(dw0.norm())


def test_router_losses_need_a_training_forward(L):
    layer, g = _layer(8, 2, 0, 1)
    with pytest.raises(ValueError, match="forward"):
        layer.router_losses(0.1)


def test_example_step_trains(L):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import rl_step
    policy = rl_step.TinyPolicy(V=1003, d=128, E=8, k=2, F=128, T_max=256)
    b = rl_step.rollout(policy, n_seqs=4, length=50, prompt=10)
    logits = policy.logits(b["tokens"], replay_kT=b["capture"])
    lp = L.moe_token_logprobs(logits, b["targets"])[0]
    assert torch.equal(lp, b["old"])                    # the replayed forward is the sampler's, bit for bit
    seen = [rl_step.step(policy, b, lr=0.2) for _ in range(6)]
    first, last = float(seen[0][0][0]), float(seen[-1][0][0])
    assert abs(float(seen[0][0][2])) < 1e-6 and last < first - 1e-3, (first, last)
    for stats, losses, counts in seen:
        assert torch.isfinite(stats).all() and torch.isfinite(losses).all()
        assert int(counts.sum()) == 4 * 40 * 2          # the scored tokens' slots
    assert L.check_status(policy.layer.dev_status) == 0
