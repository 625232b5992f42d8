"""A stack of layers that keep what their backward needs in 8 bits, on one
layer's scratch: the results of layers with their own, and the memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
E, k, d, F, T_max = 24, 3, 256, 384, 300


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def weights(seed):
    from block_scaled_fp8_router_gb300.layer import MoEWeightsFP8, quantize_weights
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    w = MoEWeightsFP8((0.1 * r(E, d)).bfloat16(), *quantize_weights((0.06 * r(E, 2 * F, d)).bfloat16(),
                                                                    (0.06 * r(E, d, F)).bfloat16()))
    w.transposed()
    return w, 1 + 0.2 * r(d)


def layer(w, scratch=None, ckpt8=True, **kw):
    from block_scaled_fp8_router_gb300.layer import MoELayerFP8, MoENorm
    return MoELayerFP8(w[0], kw.get("T_max", T_max), kw.get("k", k), 1, renorm=1, route_scale=1.5, norm=MoENorm(w[1]), ckpt8=ckpt8,
                       scratch=scratch)


def step(layers, x, dy):
    """Residual layers forward, their backward in the other order: every tensor that a layer returned."""
    got = []
    for lay in layers:
        y = lay.forward(x, train=True)
        got.append(y.clone())
        x = (x.float() + y.float()).bfloat16()
    for lay in reversed(layers):
        dn, dg, dW13, dW2 = lay.backward(dy, weight_grads=True)
        losses, counts, dr, dwr = lay.router_losses(0.1, 0.01, d_gates=dg)
        dx, dw, _ = lay.norm_backward(dn, dr, dres=dy)
        got += [t.clone() for t in (dn, dg, dW13, dW2, losses, counts, dr, dwr, dx, dw)]
        dy = dx
    return got


def test_stack_on_one_scratch(L):
    ws = [weights(s) for s in range(3)]
    g = torch.Generator(device=DEV).manual_seed(9)
    own = [layer(w) for w in ws]
    first = layer(ws[0])
    second = layer(ws[1], first)
    shared = [first, second, layer(ws[2], second)]        # of a layer that shares itself
    for T in (300, 17, 128):
        x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
        dy = (1e-2 * torch.randn(T, d, device=DEV, generator=g)).bfloat16()
        assert all(torch.equal(a, b) for a, b in zip(step(own, x, dy), step(shared, x, dy)))
    # what a layer returned stays until its own next call
    outs = [lay.forward(x, train=True) for lay in shared]
    keep = [o.clone() for o in outs]
    grads = [lay.backward(dy, weight_grads=True) for lay in shared]
    want = [lay.backward(dy, weight_grads=True) for lay in own if lay.forward(x, train=True) is not None]
    assert all(torch.equal(a, b) for a, b in zip(outs, keep))
    assert all(torch.equal(a, b) for p, q in zip(grads, want) for a, b in zip(p, q))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(shared, x, dy)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, step(own, x, dy)))


def test_memory_of_one_more_layer(L):
    """A layer on another's scratch holds what it keeps and what it returns."""
    ws = [weights(s) for s in range(3)]
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(T_max, d, device=DEV, generator=g).bfloat16()
    dy = (1e-2 * torch.randn(T_max, d, device=DEV, generator=g)).bfloat16()

    def more(scratch, w):
        at = torch.cuda.memory_allocated()
        lay = layer(w, scratch)
        lay.forward(x, train=True)
        lay.backward(dy, weight_grads=True)
        return lay, torch.cuda.memory_allocated() - at

    first, alone = more(None, ws[0])
    _second, own = more(None, ws[1])
    third, shared = more(first, ws[2])
    A = T_max * k
    kept = A * 2 * F * (1 + 4 / 128) + T_max * d * (2 + 1 + 4 / 128) + 8 * T_max + 16 * A + 4 * (2 * E + 1)
    returned = T_max * d * 2 * 2 + 4 * T_max * k + 3 * E * d * F * 4
    tensors = 24
    assert shared <= kept + returned + 512 * tensors      # the allocator's 512 bytes a tensor
    scratch = A * (d * 2 + d + d * 2 + F * 2 + 2 * F)     # the largest of it: outputs, sorted rows, the backward's rows and operands
    assert own - shared >= scratch and alone - shared >= scratch
    assert third.out_sorted is first.out_sorted


def test_refusals(L):
    w = weights(0)
    lay = layer(w)
    with pytest.raises(ValueError):
        layer(w, lay, ckpt8=False)
    with pytest.raises(ValueError):
        layer(w, layer(w, ckpt8=False))
    with pytest.raises(ValueError):
        layer(w, lay, T_max=T_max + 1)
    with pytest.raises(ValueError):
        layer(w, lay, k=k + 1)
