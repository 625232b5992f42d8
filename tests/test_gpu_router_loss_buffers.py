"""The buffers of the layer's router_losses: they stay where they are while
batches change their tokens and sequences, so that a captured graph and an
eager call can follow each other."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def _layer(T_max=400, E=40, k=3, d=256, F=128):
    from block_scaled_fp8_router_gb300.layer import MoELayerFP8, MoEWeightsFP8, quantize_weights
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = MoEWeightsFP8((0.1 * r(E, d)).bfloat16(), *quantize_weights((0.06 * r(E, 2 * F, d)).bfloat16(),
                                                                    (0.06 * r(E, d, F)).bfloat16()))
    return MoELayerFP8(w, T_max, k, 1, renorm=1, route_scale=1.5), g


def _batch(g, T, B):
    x = torch.randn(T, 256, device="cuda", generator=g).bfloat16()
    cut = torch.randint(0, T + 1, (B - 1,), device="cuda", generator=g).sort().values
    off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).int()
    return x, off, 1e-2 * torch.randn(T, 3, device="cuda", generator=g)


def test_router_losses_keep_their_buffers(L):
    """Nothing but counts moves, whatever T and B do, and the results are those of a new layer."""
    layer, g = _layer()
    seen = set()
    for T, B in ((300, 3), (400, 1), (17, 9), (130, 2), (400, 700), (1, 3), (65, 701)):
        x, off, dg = _batch(g, T, B)
        layer.forward(x, train=True)
        got = layer.router_losses(0.1, 0.01, d_gates=dg, seq_offsets=off)
        assert got[1].shape == (B, 40) and int(got[1].sum()) == T * 3
        seen.add((got[0].data_ptr(), got[2].data_ptr(), got[3].data_ptr(), layer._rl["ws"].data_ptr()))
        fresh, _ = _layer()
        fresh.forward(x, train=True)
        for a, b in zip(got, fresh.router_losses(0.1, 0.01, d_gates=dg, seq_offsets=off)):
            assert torch.equal(a, b)
    assert len(seen) == 1
    assert L.check_status(layer.dev_status) == 0


def test_router_losses_workspace_holds_every_batch(L):
    """The workspace made once is enough for each number of tokens."""
    layer, g = _layer(T_max=1000, E=200)
    x, off, dg = _batch(g, 5, 2)
    layer.forward(x, train=True)
    layer.router_losses(0.1, d_gates=dg, seq_offsets=off)
    have = layer._rl["ws"].numel()
    for T in range(0, 1001):
        assert L.moe_router_logits_workspace_size(T, 256, 200) <= have
        assert L.moe_router_backward_dense_workspace_size(T, 256, 200) <= have
    for B in (1, 65535):
        assert L.moe_balance_loss_workspace_size(1000, 200, B) <= have


def test_router_losses_graph_outlives_other_batches(L):
    """A graph captured at three sequences, replayed after eager calls with
    more, gives what it gave."""
    layer, g = _layer()
    x, off, dg = _batch(g, 300, 3)
    layer.forward(x, train=True)
    want = [t.clone() for t in layer.router_losses(0.1, 0.01, d_gates=dg, seq_offsets=off)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.router_losses(0.1, 0.01, d_gates=dg, seq_offsets=off)
    for B in (7, 500):
        _, off2, _ = _batch(g, 300, B)
        layer.router_losses(0.1, 0.01, d_gates=dg, seq_offsets=off2)
    held = [torch.full((3, 40), -1, dtype=torch.int32, device="cuda") for _ in range(64)]
    graph.replay()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert all(bool(h.eq(-1).all()) for h in held)
