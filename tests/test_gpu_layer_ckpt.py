"""The layer with a norm before it and with what its backward needs kept in
8 bits, as a training step runs them together."""
import os
import sys

import pytest
import torch

from tests import ckpt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def make(T_max=300, E=24, k=3, d=256, F=384, score=1, seed=0, norm=None, **kw):
    from block_scaled_fp8_router_gb300.layer import MoELayerFP8, MoENorm, MoEWeightsFP8, quantize_weights
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    w = MoEWeightsFP8((0.1 * r(E, d)).bfloat16(), *quantize_weights((0.06 * r(E, 2 * F, d)).bfloat16(),
                                                                    (0.06 * r(E, d, F)).bfloat16()))
    n = None
    if norm:
        n = MoENorm(1 + 0.2 * r(d), 0.1 * r(d) if norm == "ln" else None, eps=1e-5, center=norm == "ln")
    return MoELayerFP8(w, T_max, k, score, renorm=1, route_scale=1.5, norm=n, **kw), g


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("T,E,k,d,F", [(300, 24, 3, 256, 384), (1, 8, 2, 128, 128), (37, 64, 6, 512, 128), (129, 4, 4, 128, 256)])
def test_ckpt8_against_its_parts(L, T, E, k, d, F):
    """The forward to the bit as without; the backward that of the decoded
    pre-activations through the fp32 calls, but for codes at a border."""
    std, _ = make(E=E, k=k, d=d, F=F)
    lay, g = make(E=E, k=k, d=d, F=F, ckpt8=True)
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    dy = (1e-2 * torch.randn(T, d, device=DEV, generator=g)).bfloat16()
    y0 = std.forward(x, train=True).clone()
    assert torch.equal(lay.forward(x, train=True), y0)
    A = T * k
    dx, dg, dW13, dW2 = lay.backward(dy, weight_grads=True)
    dx, dg = dx.clone(), dg.clone()
    only = lay.backward(dy)
    assert torch.equal(only[0], dx) and torch.equal(only[1], dg)
    # the same steps from h in fp32
    h = R.decode(lay.h_q[:A], lay.h_s[:A]).float()
    b, off = lay._bw, lay.offsets
    dh = L.moe_swiglu_backward(b["d_act"][:A], h)
    _, _, t13q, t13s = lay.w.transposed()
    rows = L.moe_grouped_gemm_fp8(*dh, off, t13q, t13s)
    # one code in a thousand at a border, a step of it 2^-3 of the value: 2^-3 sqrt(1e-3) = 4e-3
    assert rel(dx, L.moe_dispatch_backward(rows, lay.sl2[:A], T, k)) <= 4e-3
    pad, ld = L.moe_wgrad_pad_offsets(off), L.wgrad_ld(A, E)
    q = lambda src, C, **kw: L.moe_wgrad_quant(src, off, pad, C, ld, True, sorted_to_slot=lay.s2s[:A], k=k, **kw)
    act, dhT = q(L.WGRAD_SRC_ACT, F, h=h, F=F), q(L.WGRAD_SRC_DH, 2 * F, h=h, d_act=b["d_act"], F=F)
    want2 = L.moe_wgrad_gemm(*q(L.WGRAD_SRC_GDY, d, dy=dy, gates=lay.gates[:T]), *act, pad)
    want13 = L.moe_wgrad_gemm(*dhT, *q(L.WGRAD_SRC_X, d, x=x), pad)
    assert rel(dW2, want2) <= 4e-3 and rel(dW13, want13) <= 4e-3
    # the gates' gradient by its formula, in 64 bits
    _, a64, _, e_act = R.swiglu(b["d_act"][:A], lay.h_q[:A], lay.h_s[:A])
    da, at = b["d_act"][:A].double(), lay.sl2[:A].long()
    gate = lay.gates[:T].reshape(-1).double()
    tol = ((da.abs() * e_act).sum(1) + (12 + F / 128) * R.U * (da * a64).abs().sum(1))[at] / gate
    assert bool(((dg.reshape(-1).double() - (da * a64).sum(1)[at] / gate).abs() <= tol).all())
    # and against <dy, out> of the layer that keeps its outputs: both carry E4M3 roundings of 2.6% rms of their
    # factors (act, or g dy, act's two factors), which a dot product of d terms keeps in proportion: 3 of them, 3 sigma
    dx_s, dg_s = std.backward(dy)
    if A >= 100:
        assert rel(dg, dg_s) <= 0.15 and rel(dx, dx_s) <= 0.15
    assert L.check_status(lay.dev_status) == 0


@pytest.mark.parametrize("norm", ["rms", "ln"])
@pytest.mark.parametrize("ckpt8", [False, True])
def test_norm_in_front(L, norm, ckpt8):
    lay, g = make(norm=norm, ckpt8=ckpt8)
    plain, _ = make()
    T, d, n = 211, 256, lay.norm
    x = (3 * torch.randn(T, d, device=DEV, generator=g) + 0.5).bfloat16()
    dy = (1e-2 * torch.randn(T, d, device=DEV, generator=g)).bfloat16()
    keep = x.clone()
    y = lay.forward(x, train=True).clone()
    xn, mu, r, h = R.norm(x, n.weight, n.bias, n.eps, n.center)
    got = lay.xn[:T].double()
    assert bool(((got - xn).abs() <= 2.0 ** -8 * xn.abs() + 2.0 ** -16).all())
    # The routing is that of the normalised rows; the experts' operand has one rounding less than the bf16 rows'.
    # Values 2^-9 (bf16, on average) apart, rounded to steps of up to 2^-3, differ in a code in 64: by
    # sqrt(2^-9 2^-3) = 1.6% rms at most.  act = silu(g) u has that from two factors, sqrt(2) 1.6% = 2.2%, and is
    # rounded to steps of 2^-3 again: sqrt(0.022 2^-3) = 5.2%
    y0 = plain.forward(lay.xn[:T].contiguous())
    assert torch.equal(lay.ids[:T], plain.ids[:T]) and torch.equal(lay.gates[:T], plain.gates[:T])
    assert rel(y, y0) <= 0.052
    eval_y = lay.forward(x).clone()
    assert torch.equal(eval_y, y)
    with pytest.raises(ValueError):                       # the evaluation kept nothing
        lay.backward(dy)
    with pytest.raises(ValueError):
        lay.norm_backward(dy)
    lay.forward(x, train=True)
    if ckpt8:
        x.zero_()                                         # the caller's rows are not needed any more
        h = R.decode(lay.xhat_q[:T], lay.xhat_s[:T])
    else:
        h = (x.double() - (lay.n_mean[:T].double()[:, None] if n.center else 0)) * lay.n_rstd[:T].double()[:, None]
    dn, dg = lay.backward(dy)
    _, _, dn_r, _ = lay.router_losses(0.1, 0.01, d_gates=dg)
    dx, dw, db = lay.norm_backward(dn, dn_r, dres=dy)
    rdx, rdw, rdb, size, sw, sb = R.norm_backward(dn, h, lay.n_rstd[:T], n.weight, n.center, dn_r, dy)
    assert bool(((dx.double() - rdx).abs() <= 2.0 ** -8 * rdx.abs() + 128 * R.U * size).all())
    assert bool(((dw.double() - rdw).abs() <= 64 * R.U * sw).all())
    assert (db is None) == (norm == "rms")
    if db is not None:
        assert bool(((db.double() - rdb).abs() <= 64 * R.U * sb).all())
    assert L.check_status(lay.dev_status) == 0
    del keep


def test_norm_before_the_other_forms(L):
    """The gathered form takes the same codes (the sorted form's bits); the power-of-two form quantises the normalised rows."""
    from block_scaled_fp8_router_gb300.layer import MoELayerFP8, MoEWeightsFP8, quantize_weights
    lay, g = make(norm="ln")
    gat, _ = make(norm="ln", gathered=True)
    x = (2 * torch.randn(150, 256, device=DEV, generator=g)).bfloat16()
    assert torch.equal(lay.forward(x), gat.forward(x))
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    w = MoEWeightsFP8((0.1 * r(8, 256)).bfloat16(), *quantize_weights((0.06 * r(8, 256, 256)).bfloat16(),
                                                                      (0.06 * r(8, 256, 128)).bfloat16(), ue8m0=True))
    mx = MoELayerFP8(w, 150, 2, 1, norm=lay.norm)
    y = mx.forward(x).clone()
    assert torch.equal(y, MoELayerFP8(w, 150, 2, 1).forward(mx.xn[:150].contiguous()))
    # rows of a wider buffer, and the layer with fewer rows than it was made for
    for ld in (300, 304):
        wide = torch.zeros(37, ld, dtype=torch.bfloat16, device=DEV)
        wide[:, :256] = x[:37]
        if ld % 8:                                        # the codes need rows of whole 16-byte vectors: refused
            with pytest.raises(L.MoEError):
                lay.forward(wide[:, :256])
        else:
            assert torch.equal(lay.forward(wide[:, :256]).clone(), lay.forward(x[:37].contiguous()))


def test_step_in_a_graph(L):
    """Forward, backward with weight gradients, router losses and the norm's
    backward captured once, replayed on other batches, and run eagerly in between."""
    lay, g = make(norm="ln", ckpt8=True)
    T = 200
    x = torch.empty(T, 256, dtype=torch.bfloat16, device=DEV)
    dy = torch.empty_like(x)

    def step():
        y = lay.forward(x, train=True)
        dn, dg, dW13, dW2 = lay.backward(dy, weight_grads=True)
        losses, counts, dn_r, dw_r = lay.router_losses(0.1, 0.01, d_gates=dg)
        return (y, dg, dW13, dW2, losses, counts, dw_r, *lay.norm_backward(dn, dn_r, dres=dy))

    batches = [((2 * torch.randn(T, 256, device=DEV, generator=g)).bfloat16(),
                (1e-2 * torch.randn(T, 256, device=DEV, generator=g)).bfloat16()) for _ in range(3)]

    def put(i):
        x.copy_(batches[i][0])
        dy.copy_(batches[i][1])

    want = []
    for i in range(3):
        put(i)
        want.append([t.clone() for t in step()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in (1, 0, 2):
        put(i)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, want[i]))
        put((i + 1) % 3)
        assert all(torch.equal(a, b) for a, b in zip(step(), want[(i + 1) % 3]))
    assert L.check_status(lay.dev_status) == 0


def test_replay_with_tokens_that_go_nowhere(L):
    """Tokens whose replayed ids are out of range: no rows, no gradient of their gates, the rest as ever."""
    lay, g = make(ckpt8=True, norm="rms")
    T, E, k = 90, 24, 3
    x = torch.randn(T, 256, device=DEV, generator=g).bfloat16()
    dy = torch.randn(T, 256, device=DEV, generator=g).bfloat16()
    rep = torch.rand(T, E, device=DEV, generator=g).topk(k, 1).indices.int().t().contiguous()
    rep[:, 7] = -1
    rep[1, 50] = 999
    lay.forward(x, replay_kT=rep, train=True)
    _, dg, dW13, dW2 = lay.backward(dy, weight_grads=True)
    assert L.check_status(lay.dev_status) == 1            # MOE_DEV_BAD_IDS
    lay.dev_status.zero_()
    assert not bool(dg[7].any()) and not bool(dg[50].any())
    for t in (dg, dW13, dW2):
        assert bool(t.isfinite().all())
    rep2 = torch.cat([rep[:, :7], rep[:, 8:50], rep[:, 51:]], 1).contiguous()
    keep = [i for i in range(T) if i not in (7, 50)]
    dg0 = dg[keep].clone()
    lay.forward(x[keep], replay_kT=rep2, train=True)
    assert torch.equal(lay.backward(dy[keep])[1], dg0)
    assert L.check_status(lay.dev_status) == 0


def test_refusals(L):
    with pytest.raises(ValueError):
        make(ckpt8=True, gathered=True)
    lay, g = make(norm="rms", ckpt8=True)
    dy = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        lay.norm_backward(dy)
    with pytest.raises(ValueError):
        make()[0].norm_backward(dy)
    with pytest.raises(ValueError):
        lay.forward(torch.zeros(4, 256, device=DEV), train=True)          # not bf16


@pytest.mark.parametrize("norm,ckpt8", [("rms", False), (None, True), ("rms", True)])
def test_a_forward_that_fails_keeps_nothing(L, norm, ckpt8):
    """Its norm has already written over what the forward before it kept."""
    lay, g = make(norm=norm, ckpt8=ckpt8)
    x = torch.randn(40, 256, device=DEV, generator=g).bfloat16()
    lay.forward(x, train=True)
    with pytest.raises(ValueError):
        lay.forward(x[:20], replay_kT=torch.zeros(3, 7, dtype=torch.int32, device=DEV), train=True)
    with pytest.raises(ValueError):
        lay.backward(x)
    lay.forward(x, train=True)
    dx, _ = lay.backward(x)
    assert dx.shape == x.shape


@pytest.mark.parametrize("norm,ckpt8", [(True, False), (False, True), (True, True)])
def test_example_step(L, norm, ckpt8):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import rl_step
    policy = rl_step.TinyPolicy(V=1003, d=128, E=8, k=2, F=128, T_max=256, norm=norm, ckpt8=ckpt8)
    b = rl_step.rollout(policy, n_seqs=4, length=50, prompt=10)
    for _ in range(3):
        stats, losses, counts = rl_step.step(policy, b)
        assert torch.isfinite(stats).all() and torch.isfinite(losses).all() and int(counts.sum()) == 4 * 40 * 2
    if norm:
        assert bool((policy.layer.norm.weight != 1).any()) and torch.isfinite(policy.layer.norm.weight).all()
    assert L.check_status(policy.layer.dev_status) == 0
