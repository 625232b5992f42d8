"""The norm and its backward on the GPU against 64-bit forms.

Tolerances: a sum of a row runs over at most 32 values a thread, 5 shuffles and
16 warps' parts, 53 additions of half a step of fp32 each (2^-24) relative to
the sum of magnitudes, and a handful of products: 128 half steps bound every
fp32 quantity of a row.  What is rounded to bf16 is off by 2^-8 of itself more.
"""
import pytest
import torch

from tests import ckpt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
K = 128 * R.U


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def rows_of(rows, cols, dt, g, ld=None, shift=0):
    """[rows, cols] of a buffer with row stride ld, `shift` elements in."""
    buf = torch.randn(rows * (ld or cols) + shift + 64, device=DEV, generator=g) * 2 + 0.5
    buf = buf.to(dt)
    return torch.as_strided(buf, (rows, cols), (ld or cols, 1), shift)


def check(got, ref, size, dt, what):
    err = (got.double() - ref).abs()
    tol = HALF_OF[dt] * ref.abs() + K * size
    assert bool((err <= tol).all()), (what, float((err - tol).max()), float((err / tol.clamp_min(1e-300)).max()))


HALF_OF = {torch.bfloat16: R.HALF[torch.bfloat16], torch.float32: 0.0}

SIZES = [(1, 7168), (3, 128), (5, 1), (4, 2), (7, 33), (130, 1000), (257, 2048), (19, 5000), (2, 8192), (3, 8200),
         (6, 16384), (1300, 384), (2, 16383)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("center", [True, False])
def test_forward(L, rows, cols, dt, center):
    g = torch.Generator(device=DEV).manual_seed(rows * 31 + cols)
    x = rows_of(rows, cols, dt, g)
    wdt = dt if cols % 3 else torch.float32
    w = (1 + 0.3 * torch.randn(cols, device=DEV, generator=g)).to(wdt)
    b = (0.2 * torch.randn(cols, device=DEV, generator=g)).to(wdt) if rows % 2 else None
    blocks = cols % 128 == 0
    y, mean, rstd, codes, ckpt = L.moe_layer_norm(x, w, b, eps=1e-5, center=center, mean=True, rstd=True, codes=blocks,
                                                  ckpt=blocks)
    ry, mu, r, h = R.norm(x, w, b, 1e-5, center)
    size = (h.abs() + 1) * w.double().abs() + (0 if b is None else b.double().abs())
    check(y, ry, size, dt, "y")
    check(mean, mu, mu.abs() + 1 / r, torch.float32, "mean")
    check(rstd, r, r, torch.float32, "rstd")
    if not center:
        assert bool((mean == 0).all())
    if blocks:
        for (q, s), v, sz in ((codes, ry, size), (ckpt, h, h.abs() + 1)):
            amax = v.view(rows, -1, 128).abs().amax(2)
            esz = sz.view(rows, -1, 128).amax(2)
            assert bool(((s.double() - amax / 448).abs() <= 2 * K * esz / 448).all())
            assert bool(((R.decode(q, s) - v).abs() <= R.code_error(v, s) + 2 * K * sz).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols,ld,shift", [(1000, 1008, 8), (1000, 1003, 0), (256, 256, 1), (2048, 4096, 2048)])
def test_forward_strides_and_place(L, dt, cols, ld, shift):
    """Row strides and starts with and without whole 16-byte vectors; y over x; y beside x in one buffer."""
    g = torch.Generator(device=DEV).manual_seed(cols + ld)
    x = rows_of(37, cols, dt, g, ld, shift)
    w = torch.randn(cols + 1, device=DEV, generator=g).to(dt)[1:]        # not 16-byte aligned
    ry, _, r, h = R.norm(x, w, None, 1e-3, True)
    x2 = rows_of(37, cols, dt, g, ld, shift)
    x2.copy_(x)
    y, *_ = L.moe_layer_norm(x, w, eps=1e-3)
    check(y, ry, (h.abs() + 1) * w.double().abs(), dt, "y")
    y2, *_ = L.moe_layer_norm(x2, w, eps=1e-3, y=x2)
    assert y2 is x2 and torch.equal(y2, y)
    if ld >= 2 * cols:
        both = torch.zeros(37, 2 * cols, dtype=dt, device=DEV)
        both[:, :cols] = x
        L.moe_layer_norm(both[:, :cols], w, eps=1e-3, y=both[:, cols:])
        assert torch.equal(both[:, cols:], y) and torch.equal(both[:, :cols], x)


@pytest.mark.parametrize("dt,cols,shift", [(torch.bfloat16, 4, 3), (torch.bfloat16, 1, 1), (torch.bfloat16, 6, 1),
                                           (torch.float32, 1, 1), (torch.float32, 2, 1), (torch.float32, 1, 2)])
@pytest.mark.parametrize("center", [True, False])
def test_first_row_ends_in_its_first_16_bytes(L, dt, cols, shift, center):
    """Rows shorter than the rest of the 16 bytes that the tensor starts in, on
    SMs whose shared memory holds NaN: nothing behind the row is added in."""
    g = torch.Generator(device=DEV).manual_seed(cols + 10 * shift)
    rows = 400
    x, dy = rows_of(rows, cols, dt, g, shift=shift), rows_of(rows, cols, dt, g, shift=shift)
    w = 1 + 0.3 * torch.randn(cols, device=DEV, generator=g)
    bad = torch.full((1000, 8191), float("nan"), device=DEV)
    dirty = lambda: L.moe_layer_norm(bad, bad[0], bad[0], rstd=True)[2]
    r_bad = dirty()
    y, mean, rstd, _, _ = L.moe_layer_norm(x, w, eps=1e-2, center=center, mean=True, rstd=True)
    ry, mu, r, h = R.norm(x, w, None, 1e-2, center)
    size = (h.abs() + r[:, None] * (mu.abs() if center else 0 * mu)[:, None] + 1) * w.double().abs()
    L.moe_layer_norm_backward(bad, r_bad, x=bad, weight=bad[0], center=False)
    dx, dw, db = L.moe_layer_norm_backward(dy, rstd, x=x, mean=mean, weight=w, center=center, dbias=True)
    check(mean, mu, mu.abs() + 1 / r, torch.float32, "mean")
    check(y, ry, size, dt, "y")
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    rdx, rdw, rdb, size, sw, sb = R.norm_backward(dy, h, rstd, w, center)
    check(dx, rdx, size, dt, "dx")
    assert bool(((dw.double() - rdw).abs() <= K * sw).all()) and bool(((db.double() - rdb).abs() <= K * sb).all())


@pytest.mark.parametrize("rows,cols,dt,shift", [(400, 1, torch.bfloat16, 1), (300, 5, torch.float32, 3), (211, 1001, torch.bfloat16, 2),
                                                (170, 3001, torch.float32, 1), (3, 16383, torch.float32, 1), (5, 9001, torch.bfloat16, 3)])
@pytest.mark.parametrize("center", [True, False])
def test_backward_odd_rows_with_both_additions(L, rows, cols, dt, shift, center):
    """Staged where the rows fit beside each other, in place where not; starts off a 16-byte boundary, shared memory
    that holds NaN."""
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    x, dy, res = (rows_of(rows, cols, dt, g, shift=s) for s in (shift, 0, shift))
    add = rows_of(rows, cols, torch.float32, g, shift=shift)
    w = 1 + 0.3 * torch.randn(cols, device=DEV, generator=g)
    _, mean, rstd, _, _ = L.moe_layer_norm(x, w, eps=1e-2, center=center, mean=True, rstd=True)
    bad = torch.full((1000, 8191), float("nan"), device=DEV)
    r_bad = L.moe_layer_norm(bad, bad[0], bad[0], rstd=True)[2]
    L.moe_layer_norm_backward(bad, r_bad, x=bad, weight=bad[0], center=False)
    dx, dw, db = L.moe_layer_norm_backward(dy, rstd, x=x, mean=mean, weight=w, center=center, dy_add=add, dx_add=res, dbias=True)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    rdx, rdw, rdb, size, sw, sb = R.norm_backward(dy, h, rstd, w, center, add, res)
    check(dx, rdx, size, dt, "dx")
    assert bool(((dw.double() - rdw).abs() <= K * sw).all()) and bool(((db.double() - rdb).abs() <= K * sb).all())


def test_forward_far_mean_and_constant_rows(L):
    """A mean a thousand times the spread; a constant row is 0 before the bias; scale of the RMS form."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(64, 4096, device=DEV, generator=g) + 1000.0
    x[7] = 3.25
    y, mean, rstd, _, _ = L.moe_layer_norm(x, None, None, eps=1e-5, mean=True, rstd=True)
    ry, mu, r, h = R.norm(x, None, None, 1e-5, True)
    keep = torch.arange(64, device=DEV) != 7
    # x - mu' is exact to half a step of itself; what the first mean lacks is taken out
    check(y[keep], ry[keep], h[keep].abs() + 1, torch.float32, "y")
    assert bool((y[7] == 0).all()) and float(mean[7]) == 3.25
    assert abs(float(rstd[7]) * 1e-5 ** 0.5 - 1) < 1e-6
    b = torch.randn(4096, device=DEV, generator=g)
    assert torch.equal(L.moe_layer_norm(x, None, b)[0][7], b)


@pytest.mark.parametrize("center", [True, False])
def test_forward_infinities_and_large_values(L, center):
    """Infinities and NaN stay in their row; values whose squares leave fp32 give r = 0."""
    x = torch.randn(6, 512, device=DEV)
    clean = x.clone()
    x[1, 3], x[2, 500], x[4] = float("inf"), float("nan"), 1e30
    y, _, rstd, codes, _ = L.moe_layer_norm(x, center=center, mean=True, rstd=True, codes=True, ckpt=True)
    ref, _, _, rcodes, _ = L.moe_layer_norm(clean, center=center, mean=True, rstd=True, codes=True, ckpt=True)
    for i in (0, 3, 5):
        assert torch.equal(y[i], ref[i]) and torch.equal(codes[0][i], rcodes[0][i])
    assert bool(y[2].isnan().all()) and bool(y[1].isnan().any())
    if not center:
        assert float(rstd[4]) == 0.0 and bool((y[4] == 0).all())


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", ["x", "ckpt", "all"])
def test_backward(L, rows, cols, dt, mode):
    if mode == "ckpt" and cols % 128:
        pytest.skip("codes are blocks of 128")
    center = (rows + cols) % 2 == 0
    g = torch.Generator(device=DEV).manual_seed(rows * 7 + cols)
    x = rows_of(rows, cols, dt, g)
    dy = rows_of(rows, cols, dt, g)
    w = (1 + 0.3 * torch.randn(cols, device=DEV, generator=g)).to(dt)
    add = torch.randn(rows, cols, device=DEV, generator=g) if mode == "all" else None
    dres = rows_of(rows, cols, dt, g) if mode == "all" else None
    eps = 0.5 if cols <= 2 else 1e-5
    blocks = mode == "ckpt"
    _, mean, rstd, _, ckpt = L.moe_layer_norm(x, w, eps=eps, center=center, mean=center, rstd=True, ckpt=blocks)
    if blocks:
        h = R.decode(*ckpt)
    else:
        h = (x.double() - (mean.double()[:, None] if center else 0)) * rstd.double()[:, None]
    dx, dw, db = L.moe_layer_norm_backward(dy, rstd, x=None if blocks else x, mean=mean, ckpt=ckpt, weight=w,
                                           center=center, dy_add=add, dx_add=dres, dbias=True)
    rdx, rdw, rdb, size, sw, sb = R.norm_backward(dy, h, rstd, w, center, add, dres)
    check(dx, rdx, size, dt, "dx")
    # a column's sum: a group's rows, 8 groups, 8 runs of up to 19 parts
    n = (rows // 100 + 64) * R.U
    assert bool(((dw.double() - rdw).abs() <= n * sw + 1e-30).all())
    assert bool(((db.double() - rdb).abs() <= n * sb + 1e-30).all())


@pytest.mark.parametrize("rows,cols,dt,ld", [(6000, 5000, torch.bfloat16, 5000), (5000, 4097, torch.float32, 4097),
                                             (5000, 4097, torch.bfloat16, 4099), (30000, 130, torch.bfloat16, 130),
                                             (3000, 16000, torch.float32, 16000), (30000, 128, torch.float32, 128)])
def test_many_rows(L, rows, cols, dt, ld):
    """Rows enough that every group goes through its stages many times, forward and backward."""
    g = torch.Generator(device=DEV).manual_seed(cols)
    x, dy = rows_of(rows, cols, dt, g, ld), rows_of(rows, cols, dt, g, ld)
    w, b = torch.randn(cols, device=DEV, generator=g), torch.randn(cols, device=DEV, generator=g)
    for center in (True, False):
        y, mean, rstd, _, _ = L.moe_layer_norm(x, w, b, center=center, mean=True, rstd=True)
        dx, dw, db = L.moe_layer_norm_backward(dy, rstd, x=x, mean=mean, weight=w, center=center, dbias=center)
        tw = tb = sw = sb = 0
        for r in range(0, rows, 1000):
            s = slice(r, min(rows, r + 1000))
            ry, _, rr, h = R.norm(x[s], w, b, 1e-5, center)
            check(y[s], ry, (h.abs() + 1) * w.double().abs() + b.double().abs(), dt, "y")
            h = (x[s].double() - (mean[s].double()[:, None] if center else 0)) * rstd[s].double()[:, None]
            rdx, rdw, rdb, size, aw, ab = R.norm_backward(dy[s], h, rstd[s], w, center)
            check(dx[s], rdx, size, dt, "dx")
            tw, tb, sw, sb = tw + rdw, tb + rdb, sw + aw, sb + ab
        n = (rows // 100 + 64) * R.U
        assert bool(((dw.double() - tw).abs() <= n * sw).all())
        if center:
            assert bool(((db.double() - tb).abs() <= n * sb).all())


def test_backward_place_strides_and_parts(L):
    """dx over dy and over dx_add; strided rows; each output alone gives the same bits."""
    g = torch.Generator(device=DEV).manual_seed(3)
    rows, cols = 700, 520
    for dt, ld, shift in ((torch.bfloat16, 528, 8), (torch.bfloat16, 523, 3), (torch.float32, 521, 1)):
        x, dy = rows_of(rows, cols, dt, g, ld, shift), rows_of(rows, cols, dt, g, ld, shift)
        w = torch.randn(cols, device=DEV, generator=g)
        _, mean, rstd, _, _ = L.moe_layer_norm(x, w, mean=True, rstd=True)
        kw = dict(x=x, mean=mean, weight=w)
        dx, dw, db = L.moe_layer_norm_backward(dy, rstd, dbias=True, **kw)
        rdx, rdw, rdb, size, _, _ = R.norm_backward(dy, (x.double() - mean.double()[:, None]) * rstd.double()[:, None],
                                                    rstd, w, True)
        check(dx, rdx, size, dt, "dx")
        assert torch.equal(L.moe_layer_norm_backward(dy, rstd, dweight=False, **kw)[0], dx)
        assert torch.equal(L.moe_layer_norm_backward(dy, rstd, dx=False, **kw)[1], dw)
        assert torch.equal(L.moe_layer_norm_backward(dy, rstd, dx=None, dweight=False, dbias=True, **kw)[2], db)
        res = rows_of(rows, cols, dt, g, ld, shift)
        with_res = L.moe_layer_norm_backward(dy, rstd, dx_add=res, **kw)[0].clone()
        assert torch.equal(L.moe_layer_norm_backward(dy, rstd, dx_add=res, dx=res, **kw)[0], with_res)
        over = torch.as_strided(torch.empty(rows * ld + shift, dtype=dt, device=DEV), (rows, cols), (ld, 1), shift)
        over.copy_(dy)
        assert torch.equal(L.moe_layer_norm_backward(over, rstd, dx=over, **kw)[0], dx)


@pytest.mark.parametrize("center", [True, False])
def test_backward_against_differences(L, center):
    """d sum(c y) along random directions of x, weight and bias: central differences of the forward."""
    g = torch.Generator(device=DEV).manual_seed(11)
    rows, cols, h = 9, 96, 4e-3
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    x, c, w, b = r(rows, cols), r(rows, cols), 1 + 0.2 * r(cols), r(cols)
    _, mean, rstd, _, _ = L.moe_layer_norm(x, w, b, center=center, mean=True, rstd=True)
    dx, dw, db = L.moe_layer_norm_backward(c, rstd, x=x, mean=mean, weight=w, center=center, dbias=True)
    f = lambda x, w, b: float((c.double() * L.moe_layer_norm(x, w, b, center=center)[0].double()).sum())
    for v, grad, at in ((r(rows, cols), dx, 0), (r(cols), dw, 1), (r(cols), db, 2)):
        args = [x, w, b]
        hi = args[:at] + [args[at] + h * v] + args[at + 1:]
        lo = args[:at] + [args[at] - h * v] + args[at + 1:]
        d = (f(*hi) - f(*lo)) / (2 * h)
        # truncation h^2 / 6 of a third derivative of a few times the first's size; rounding 2^-24 sum |c y| / h
        tol = 1e-3 * float((grad.double() * v.double()).norm()) + 2 * R.U * float(c.abs().sum()) * 4 / h
        assert abs(d - float((grad.double() * v.double()).sum())) <= tol, at


def test_empty_and_unwritten(L):
    w = torch.ones(256, device=DEV)
    y, mean, rstd, codes, ckpt = L.moe_layer_norm(torch.empty(0, 256, device=DEV), w, mean=True, rstd=True, codes=True, ckpt=True)
    assert y.shape == (0, 256) and codes[0].shape == (0, 256)
    dx, dw, db = L.moe_layer_norm_backward(torch.empty(0, 256, device=DEV), rstd, x=y, mean=mean, weight=w, dbias=True,
                                           dweight=torch.full((256,), 7.0, device=DEV))
    assert dx.shape == (0, 256) and not bool(dw.any()) and not bool(db.any())
    # only the rows given are written
    buf = torch.full((10, 264), 5.0, device=DEV)
    x = torch.randn(4, 256, device=DEV)
    L.moe_layer_norm(x, w, y=buf[2:6, :256])
    assert bool((buf[:2] == 5).all()) and bool((buf[6:] == 5).all()) and bool((buf[2:6, 256:] == 5).all())


def test_streams_and_graph(L):
    """The same bits on a side stream, and in a captured graph replayed on other data."""
    g = torch.Generator(device=DEV).manual_seed(2)
    x, dy = torch.randn(300, 1024, device=DEV, generator=g).bfloat16(), torch.randn(300, 1024, device=DEV, generator=g).bfloat16()
    w = torch.randn(1024, device=DEV, generator=g)

    def both(stream=None):
        y, mean, rstd, codes, ckpt = L.moe_layer_norm(x, w, mean=True, rstd=True, codes=True, ckpt=True, stream=stream)
        return (y, *codes, *ckpt, *L.moe_layer_norm_backward(dy, rstd, ckpt=ckpt, weight=w, dbias=True, stream=stream))

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    keep = (x.clone(), dy.clone())
    x.copy_(dy)
    dy.copy_(keep[0])
    graph.replay()
    swapped = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(swapped, both()))
    x.copy_(keep[0])
    dy.copy_(keep[1])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_refusals(L):
    x = torch.randn(8, 256, device=DEV)
    with pytest.raises(L.MoEError):                                     # codes of a row that is no whole blocks
        L.moe_layer_norm(x[:, :200].contiguous(), codes=True)
    with pytest.raises(L.MoEError):                                     # codes need whole vectors
        L.moe_layer_norm(torch.randn(8 * 257 + 1, device=DEV)[1:].view(8, 257)[:, :256], codes=True)
    with pytest.raises(L.MoEError):                                     # y over x one row on
        buf = torch.randn(9, 256, device=DEV)
        L.moe_layer_norm(buf[:8], y=buf[1:])
    with pytest.raises(L.MoEError):
        L.moe_layer_norm(torch.randn(2, 16385, device=DEV))
    with pytest.raises(L.MoEError):
        L.moe_layer_norm(x, eps=-1.0)
    with pytest.raises(TypeError):
        L.moe_layer_norm(x.half())
    with pytest.raises(TypeError):
        L.moe_layer_norm(x, torch.ones(256, device=DEV), torch.ones(256, device=DEV).bfloat16())
    with pytest.raises(ValueError):
        L.moe_layer_norm(x, torch.ones(255, device=DEV))
    rstd = torch.ones(8, device=DEV)
    with pytest.raises(ValueError):
        L.moe_layer_norm_backward(x, rstd)                              # neither x nor ckpt
    with pytest.raises(ValueError):
        L.moe_layer_norm_backward(x, rstd, x=x)                         # center without mean
    with pytest.raises(ValueError):
        L.moe_layer_norm_backward(x, rstd, x=x, center=False, dx=False, dx_add=x)
    with pytest.raises(L.MoEError):
        buf = torch.randn(9, 256, device=DEV)
        L.moe_layer_norm_backward(buf[:8], rstd, x=x, center=False, dx=buf[1:])
    with pytest.raises(L.MoEError):
        L.moe_layer_norm_backward(x, rstd, x=x, center=False, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
