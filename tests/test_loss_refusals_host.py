"""Calls of the training-step losses that are refused on the host, before any
CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


SHAPE, UNSUPPORTED = 2, 6
BASE = 0x100000


def _at(off):
    return ctypes.c_void_p(BASE + off)


def _logprobs(L, N=4, tau=1.0, logprobs=_at(0x3000)):
    return L._lib.moe_token_logprobs(_at(0), 1, N, 64, 64, _at(0x2000), 64, tau, logprobs, None, None, None)


def _policy(L, N=4, V=64, ld=64, ldd=64, tau=1.0, bits=64, logits=_at(0), targets=_at(0x2000), old=_at(0x3000),
            adv=_at(0x4000), ref=_at(0x5000), w=_at(0x6000), stats=_at(0x7000), logprobs=_at(0x8000), d=_at(0x9000),
            work=_at(0x20000)):
    return L._lib.moe_policy_loss(logits, 1, N, V, ld, targets, bits, old, adv, ref, w, tau, 0.2, 0.2, 0.0, 0.0, 0.0, 1.0,
                                  stats, logprobs, d, ldd, work, 1 << 20, None, None)


@pytest.mark.parametrize("tau", [4.2e-39, 1e-45, 0.0, -1.0, float("inf"), float("nan")])
def test_temperatures_without_a_scale(L, tau):
    """log2(e) / temperature has to be finite in fp32: every row would be NaN."""
    assert _logprobs(L, tau=tau) == SHAPE and _policy(L, tau=tau) == SHAPE
    assert _logprobs(L, N=0, tau=tau) == SHAPE
    assert _logprobs(L, N=0, tau=4.3e-39) == 0


@pytest.mark.parametrize("T,k", [((1 << 31) - 1, 1), ((1 << 31) - 1024, 1), ((1 << 30) - 1, 2), ((1 << 28) - 500, 8)])
def test_balance_loss_token_limit(L, T, k):
    """Token numbers stay below 2^31 when a kernel steps past the last one."""
    size = L.moe_balance_loss_workspace_size(T, 8, 1)
    assert L._lib.moe_balance_loss(_at(0), _at(0), None, None, T, 8, k, 1, 0, 1, 1.0, 0.1, 0.0, 1.0, None, _at(0), _at(0),
                                   _at(0), _at(0), size, None, None) == SHAPE


@pytest.mark.parametrize("name,off", [("old", 0x3000), ("adv", 0x4000), ("ref", 0x5000), ("w", 0x6000), ("targets", 0x2000)])
def test_policy_logprobs_over_an_input(L, name, off):
    """A row's CTAs read its numbers while one of them writes its log-probability."""
    size = 32 if name == "targets" else 16
    for d in (0, 4, size - 4, -12):
        assert _policy(L, logprobs=_at(off + d)) == UNSUPPORTED, d
    assert _policy(L, targets=_at(0x2000), bits=32, logprobs=_at(0x200c)) == UNSUPPORTED


def test_policy_gradient_across_the_logits(L):
    """Row on row is the one overlap that is taken; rows between rows are none.
    (N = 4, V = 64, fp32.  The workspace comes after this check: a call that is
    refused for having none is one whose rows are taken.)"""
    taken = 4                                                 # MOE_ERR_WORKSPACE

    def call(**kw):
        return _policy(L, work=None, **kw)
    assert call(d=_at(0)) == taken and call(d=_at(0), ld=80, ldd=80) == taken
    for off in (256, 4, 252, -4, -256, 512):                  # by whole rows, by elements
        assert call(logits=_at(0x1000), d=_at(0x1000 + off)) == UNSUPPORTED, off
    assert call(d=_at(0), ld=64, ldd=80) == UNSUPPORTED
    assert call(N=1, d=_at(0), ld=64, ldd=80) == taken
    assert call(N=1, d=_at(0x40)) == UNSUPPORTED
    # gradient and logits in the halves of one buffer of 128 columns
    assert call(d=_at(256), ld=128, ldd=128) == taken and call(d=_at(252), ld=128, ldd=128) == UNSUPPORTED
    assert call(d=_at(256), ld=127, ldd=127) == UNSUPPORTED
    assert call(logits=_at(256), d=_at(0), ld=128, ldd=128) == taken
    assert call(d=_at(1024)) == taken                         # behind the last row
    assert call(d=None) == taken
