"""Calls on a stream other than the current one that make their own workspace:
what the current stream allocates after the call returns, while the other
stream is still busy, may not be that workspace's memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def _calls(L):
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    T, d, E, k, V = 700, 512, 64, 4, 3001
    x, w, dl = r(T, d).bfloat16(), (0.05 * r(E, d)).bfloat16(), r(T, E)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int()
    off = torch.tensor([0, 100, 450, T], dtype=torch.int32, device="cuda")
    z, y = r(T, V), torch.randint(0, V, (T,), device="cuda", generator=g)
    old, adv, wt = r(T) - 8, r(T), torch.rand(T, device="cuda", generator=g) + 0.1
    return {
        "policy": (lambda s: L.moe_policy_loss(z, y, old, adv, weights=wt, stream=s),
                   L.moe_policy_loss_workspace_size(T, V)),
        "balance": (lambda s: L.moe_balance_loss(dl, ids, L.MOE_SCORE_SIGMOID, 0.1, z_coef=0.01, seq_offsets=off, stream=s),
                    L.moe_balance_loss_workspace_size(T, E, 3)),
        "logits": (lambda s: (L.moe_router_logits(x, w, stream=s),), L.moe_router_logits_workspace_size(T, d, E)),
        "backward": (lambda s: L.moe_router_backward_dense(x, w, dl, stream=s),
                     L.moe_router_backward_dense_workspace_size(T, d, E)),
        "dispatch": (lambda s: L.moe_dispatch(ids, E, rows=x, stream=s), L.moe_dispatch_workspace_size(T, E, k)),
    }


@pytest.mark.parametrize("name", ["policy", "balance", "logits", "backward", "dispatch"])
def test_workspace_belongs_to_the_calls_stream(L, name, monkeypatch):
    call, size = _calls(L)[name]
    assert size > 0
    want = [t for t in call(None) if t is not None]
    made = []
    empty = L._empty

    def note(shape, dtype, like):
        t = empty(shape, dtype, like)
        if dtype == torch.uint8:
            made.append(t.data_ptr())
        return t
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    monkeypatch.setattr(L, "_empty", note)
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)             # tens of milliseconds before the call's work begins
    got = [t for t in call(side) if t is not None]
    monkeypatch.undo()
    junk = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(16)]
    assert len(made) == 1 and made[0] not in [j.data_ptr() for j in junk]
    torch.cuda.synchronize()
    for a, b in zip(want, got, strict=True):
        assert torch.equal(a, b)
    assert all(bool(j.eq(0xFF).all()) for j in junk)
