"""Refusals of the loss entry points, on the CPU: the library's host-side
checks (they return before any CUDA call) and the binding's."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


X = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)
Y = ctypes.c_void_p(0x1008)
N_ = None
BIG = 1 << 40


def test_token_logprobs_refusals(L):
    def call(logits=X, dt=0, N=4, V=64, ld=64, targets=X, bits=64, tau=1.0, lp=X):
        return L._lib.moe_token_logprobs(logits, dt, N, V, ld, targets, bits, tau, lp, N_, N_, N_)
    assert call(N=-1) == 2 and call(V=0) == 2 and call(N=1 << 28) == 2 and call(V=1 << 31, ld=1 << 31) == 2
    assert call(ld=63) == 2 and call(dt=2) == 2 and call(bits=16) == 2
    for tau in (0.0, -1.0, float("inf"), float("nan")):
        assert call(tau=tau) == 2
    assert call(logits=N_) == 1 and call(targets=N_) == 1 and call(lp=N_) == 1
    assert call(logits=ODD) == 3 and call(dt=1, logits=ctypes.c_void_p(0x1002)) == 3
    assert call(targets=ctypes.c_void_p(0x1004)) == 3
    assert call(N=0, logits=N_, targets=N_, lp=N_) == 0


def test_policy_loss_refusals(L):
    ws = L.moe_policy_loss_workspace_size(4, 64)
    assert ws > 0

    def call(logits=X, dt=1, N=4, V=64, ld=64, targets=X, bits=64, old=X, adv=X, ref=N_, w=N_, tau=1.0, lo=0.2, hi=0.2,
             beta=0.0, eta=0.0, norm=0.0, gs=1.0, stats=X, lp=X, d=X, ldd=64, work=X, wb=ws):
        return L._lib.moe_policy_loss(logits, dt, N, V, ld, targets, bits, old, adv, ref, w, tau, lo, hi, beta, eta, norm,
                                      gs, stats, lp, d, ldd, work, wb, N_, N_)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(lo=nan), dict(hi=inf), dict(beta=nan), dict(eta=inf), dict(norm=nan), dict(gs=inf), dict(lo=-0.1),
               dict(hi=-0.1), dict(norm=-1.0), dict(ldd=63), dict(tau=0.0), dict(V=0), dict(ld=10), dict(dt=7)):
        assert call(**kw) == 2, kw
    for kw in (dict(stats=N_), dict(old=N_), dict(adv=N_), dict(logits=N_), dict(targets=N_)):
        assert call(**kw) == 1, kw
    assert call(wb=ws - 1) == 4 and call(work=N_) == 4
    assert call(work=Y) == 3 and call(d=ctypes.c_void_p(0x1002)) == 3 and call(logits=ctypes.c_void_p(0x1002)) == 3


def test_router_dense_refusals(L):
    lib = L._lib
    for f, size in ((lambda T=8, d=128, E=8, x=X, w=X, o=X, ws=X, wb=BIG: lib.moe_router_logits(
                        x, w, T, d, E, o, ws, wb, N_, N_), L.moe_router_logits_workspace_size(8, 128, 8)),
                    (lambda T=8, d=128, E=8, x=X, w=X, o=X, ws=X, wb=BIG: lib.moe_router_backward_dense(
                        x, w, X, T, d, E, o, X, ws, wb, N_, N_),
                     L.moe_router_backward_dense_workspace_size(8, 128, 8))):
        assert f(T=-1) == 2 and f(d=100) == 2 and f(d=0) == 2 and f(E=0) == 2 and f(E=1025) == 2
        assert f(x=N_) == 1 and f(w=N_) == 1
        assert f(x=Y) == 3 and f(w=Y) == 3 and f(ws=Y) == 3
        assert size > 0 and f(wb=size - 1) == 4 and f(ws=N_) == 4
    assert lib.moe_router_logits(X, X, 8, 128, 8, N_, X, BIG, N_, N_) == 1
    assert lib.moe_router_logits(N_, N_, 0, 128, 8, N_, N_, 0, N_, N_) == 0
    assert lib.moe_router_backward_dense(X, X, X, 8, 128, 8, Y, X, X, BIG, N_, N_) == 3        # dx
    assert lib.moe_router_backward_dense(X, X, X, 8, 128, 8, X, Y, X, BIG, N_, N_) == 3        # dW_r
    assert lib.moe_router_backward_dense(X, X, N_, 8, 128, 8, X, X, X, BIG, N_, N_) == 1
    assert lib.moe_router_backward_dense(X, X, X, 8, 128, 8, N_, N_, N_, 0, N_, N_) == 0       # nothing asked for
    assert lib.moe_router_backward_dense(N_, N_, N_, 0, 128, 8, N_, N_, N_, 0, N_, N_) == 0


def test_balance_loss_refusals(L):
    ws = L.moe_balance_loss_workspace_size(8, 8, 2)

    def call(l=X, ids=X, mask=N_, off=X, T=8, E=8, k=2, B=2, fn=0, renorm=1, rs=1.0, a=0.1, z=0.0, gs=1.0, dg=N_, c=X,
             lo=X, d=X, work=X, wb=ws):
        return L._lib.moe_balance_loss(l, ids, mask, off, T, E, k, B, fn, renorm, rs, a, z, gs, dg, c, lo, d, work, wb, N_,
                                       N_)
    nan = float("nan")
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=33), dict(B=0), dict(B=65536),
               dict(off=N_), dict(fn=2), dict(rs=nan), dict(a=nan), dict(z=nan), dict(gs=float("inf")),
               dict(T=1 << 30, k=2)):
        assert call(**kw) == 2, kw
    for kw in (dict(l=N_), dict(ids=N_), dict(c=N_), dict(lo=N_)):
        assert call(**kw) == 1, kw
    assert call(wb=ws - 1) == 4 and call(work=N_) == 4 and call(work=Y) == 3


def test_binding_refusals(L):
    x, y, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        L.moe_token_logprobs(x, y)
    with pytest.raises(TypeError, match="logits: expected"):
        L.moe_token_logprobs(x.half(), y)
    with pytest.raises(ValueError, match="2-D"):
        L.moe_policy_loss(x[0], y, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        L.moe_policy_loss(x, y, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        L.moe_balance_loss(x, torch.zeros(4, 2, dtype=torch.int32), 0, 0.1)
    with pytest.raises(TypeError, match="logits: expected"):
        L.moe_balance_loss(x.bfloat16(), torch.zeros(4, 2, dtype=torch.int32), 0, 0.1)
    xb, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.moe_router_logits(xb, w)
    with pytest.raises(ValueError, match="CUDA"):
        L.moe_router_backward_dense(xb, w, torch.zeros(4, 8))
