"""The codes of computed values by their rule, from values that another output
of the call gives in fp32: scales amax / 448 to the bit (1 where that is 0, not
below 2^-126), codes of the product with the scale's reciprocal."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def by_rule(v):
    """Codes, scales and which scales have a reciprocal that the rule fixes to the bit (all but a mantissa of ones)."""
    b = v.view(v.shape[0], -1, 128)
    # a tensor as divisor: torch divides by a Python number through its reciprocal
    s = b.abs().amax(2) / torch.full((1, 1), 448.0, device=DEV)
    s = torch.where(s == 0, torch.ones_like(s), s.clamp_min(2.0 ** -126))
    q = (b * (torch.ones_like(s) / s)[..., None]).clamp(-448, 448).view(v.shape).to(F8).view(torch.uint8)
    fixed = (s.view(torch.int32) & 0x7FFFFF) != 0x7FFFFF
    return q, s, fixed.repeat_interleave(128, 1)


@pytest.mark.parametrize("rows,cols", [(3, 1024), (700, 7168), (400, 16384)])
@pytest.mark.parametrize("center", [True, False])
def test_norm(L, rows, cols, center):
    """Rows of any size, and weights of any: y in fp32 is what its codes are formed from, and without a weight xhat is y."""
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x = torch.randn(rows, cols, device=DEV, generator=g) * (0.1 + 10 * torch.rand(rows, 1, device=DEV, generator=g))
    w = torch.randn(cols, device=DEV, generator=g)
    # columns' blocks from the largest numbers to none at all: 1e35, 1, subnormal scales, values that are subnormal, quotients that are 0
    for at, size in enumerate((1e35, 1.0, 1e-30, 3e-36, 1e-38, 1e-42, 0.0, 2e-44)):
        w[at * 128:(at + 1) * 128] *= size
    y, _, _, codes, _ = L.moe_layer_norm(x, w, center=center, codes=True)
    q, s, fixed = by_rule(y)
    assert torch.equal(codes[1], s)
    assert torch.equal(codes[0][fixed] & 0x7F, q[fixed] & 0x7F)      # the sign of a zero is not the rule's
    assert torch.equal(codes[0][(q & 0x7F) != 0] & 0x80, q[(q & 0x7F) != 0] & 0x80)
    y, _, _, codes, ckpt = L.moe_layer_norm(x, center=center, codes=True, ckpt=True)
    q, s, fixed = by_rule(y)
    for a, b in (codes, ckpt):
        assert torch.equal(b, s) and torch.equal(a[fixed], q[fixed])


def test_infinite_scales(L):
    """An infinity makes its block's scale infinite, its code NaN and the others' zero."""
    x = torch.randn(4, 256, device=DEV)
    w = torch.ones(256, device=DEV)
    w[5] = float("inf")
    _, _, _, (q, s), _ = L.moe_layer_norm(x, w, center=False, codes=True)
    assert bool(s[:, 0].isinf().all()) and bool(s[:, 1].isfinite().all())
    q = q & 0x7F
    assert bool((q[:, 5] == 0x7F).all()) and not bool(q[:, :5].any()) and not bool(q[:, 6:128].any())
