"""The norm and its backward at the most rows the calls take."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
ROWS, PERIOD = 2 ** 31 - 1, 1 << 20


def test_most_rows():
    """2^31 - 1 rows of one column, the same 2^20 over and over: every run of
    them as the first one, that one against 64 bits, and the sums over all rows."""
    from block_scaled_fp8_router_gb300 import moe_r3 as L
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device=DEV).manual_seed(0)
    many = lambda t: t.repeat(-(-ROWS // PERIOD))[:ROWS]  # noqa: E731
    x1 = (0.5 + torch.rand(PERIOD, device=DEV, generator=g)).bfloat16()
    dy1 = torch.randn(PERIOD, device=DEV, generator=g).bfloat16()
    x, dy = many(x1)[:, None], many(dy1)[:, None]
    eps = 0.5
    y, _, rstd, _, _ = L.moe_layer_norm(x, eps=eps, center=False, rstd=True)
    r = 1.0 / (x1.double() ** 2 + eps).sqrt()
    assert bool(((rstd[:PERIOD].double() - r).abs() <= 16 * U * r).all())
    want = x1.double() * r
    assert bool(((y[:PERIOD, 0].double() - want).abs() <= (2.0 ** -8 + 32 * U) * want).all())
    dx, dw, _ = L.moe_layer_norm_backward(dy, rstd, x=x, center=False)
    h = x1.double() * rstd[:PERIOD].double()
    a = dy1.double()
    want = rstd[:PERIOD].double() * (a - h * a * h)
    size = rstd[:PERIOD].double() * (a.abs() + (h * a * h).abs())
    assert bool(((dx[:PERIOD, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 32 * U * size).all())
    for t in (y[:, 0], rstd, dx[:, 0]):
        for at in range(0, ROWS, PERIOD):
            run = t[at:at + PERIOD]
            assert torch.equal(run, t[:run.numel()])
    n, rest = divmod(ROWS, PERIOD)
    total = n * (a * h).sum() + (a * h)[:rest].sum()
    size = n * (a * h).abs().sum() + (a * h)[:rest].abs().sum()
    # a group of warps adds its rows one after another in fp32: eight groups an SM
    steps = ROWS / (8 * L.moe_device_sm_count()) + 64
    assert abs(float(dw[0].double() - total)) <= steps * U * float(size)
