"""The SwiGLU backward from 8 bits where its values are next to the smallest
numbers of fp32: scales at their floor, codes as far off as the roundings say."""
import pytest
import torch

from tests import ckpt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FLOOR = 2.0 ** -126
# a product or sum below 2^-126 is off by half of 2^-149; of dh's there are two in a row, (a u) and the product with
# the slope (at most 1.1 times as large), of act one: below 2^-148 together
TINY = 2.0 ** -148


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


@pytest.mark.parametrize("size", [1e-38, 3e-40, 1e-36])
def test_subnormal_gradients(L, size):
    A, F = 256, 128
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    h = 1.5 * r(A, 2 * F) * (0.2 + 3 * torch.rand(A, 1, device=DEV, generator=g))
    h_s = h.view(A, -1, 128).abs().amax(2) / 448.0
    h_q = (h.view(A, -1, 128) / h_s[..., None]).view(A, 2 * F).to(torch.float8_e4m3fn).view(torch.uint8)
    d_act = (size * r(A, F).double()).bfloat16()
    d_act[7] = 0
    offs = torch.tensor([0, 150, 256], dtype=torch.int32, device=DEV)
    pad = L.moe_wgrad_pad_offsets(offs)
    P = int(pad[-1])
    dh, _, dhT, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=offs, pad=pad, ld=P, dhT=True)
    v, _, e, _ = R.swiglu(d_act, h_q, h_s)
    assert float(v.abs().median()) < 1e3 * FLOOR
    pv, pe = (R.padded(t, [0, 150, 256], pad.tolist(), P) for t in (v, e))
    row = lambda t: t.view(A, -1, 128).amax(2)  # noqa: E731
    col = lambda t: t.view(P // 128, 128, -1).amax(1)  # noqa: E731
    for q, s, val, err, axis, top in ((*dh, v, e, 1, row), (dhT[0].t(), dhT[1], pv, pe, 0, col)):
        # scales: the floor or the quotient, as far off as the largest value may be; 1 for a block of zeros
        amax, emax = top(val.abs()), top(err) + TINY
        want = torch.where(amax == 0, torch.ones_like(amax), (amax / 448).clamp_min(FLOOR))
        assert bool(((s.double() - want).abs() <= 2 * emax / 448 + R.U * want).all())
        low = (amax > 0) & ((amax + 2 * emax) / 448 < FLOOR)
        assert bool((s[low] == FLOOR).all()) and (size > 1e-37 or bool(low.any()))
        # codes: half a step of the value, or of the smallest codes, and the value's own roundings
        off = (R.decode(q, s, axis) - val).abs()
        assert bool((off <= R.code_error(val, s, axis) + 2 * err + TINY).all())
        # which is far below the values themselves, so that zeros would not pass
        assert float((off > 0.5 * val.abs()).double().mean()) < 0.5 and bool((q & 0x7F).any())
