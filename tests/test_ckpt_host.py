"""What the norm and the 8-bit checkpoint calls refuse on the host, before
anything is launched (fake pointers, no GPU)."""
import ctypes

import pytest

SHAPE, NULL, ALIGN, WORKSPACE, UNSUPPORTED = 2, 1, 3, 4, 6
x, y, z, m, o = (ctypes.c_void_p(v) for v in (0x100000, 0x900000, 0x1100000, 0x100008, 0x100001))


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3._lib


def norm(lib, x_=x, dt=0, rows=4, cols=256, ld=256, w=None, b=None, wd=0, eps=1e-5, y_=y, ldy=256, yq=None, ys=None, hq=None,
         hs=None):
    return lib.moe_layer_norm(x_, dt, rows, cols, ld, w, b, wd, eps, 1, y_, ldy, None, None, yq, ys, hq, hs, None)


def test_norm(lib):
    assert norm(lib, rows=0, x_=None, y_=None) == 0
    for kw in (dict(cols=0), dict(cols=16385, ld=16385, ldy=16385), dict(rows=-1), dict(rows=1 << 31), dict(ld=255),
               dict(ldy=255), dict(dt=2), dict(wd=-1), dict(eps=-1e-3), dict(eps=float("inf")), dict(eps=float("nan")),
               dict(cols=200, yq=z, ys=z), dict(cols=200, hq=z, hs=z)):
        assert norm(lib, **kw) == SHAPE, kw
    for kw in (dict(x_=None), dict(y_=None), dict(yq=z), dict(ys=z), dict(hq=z), dict(hs=z)):
        assert norm(lib, **kw) == NULL, kw
    for kw in (dict(x_=o), dict(y_=o), dict(w=o), dict(b=ctypes.c_void_p(0x2), wd=1), dict(x_=m, yq=z, ys=z),
               dict(ld=260, yq=z, ys=z), dict(yq=o, ys=z), dict(w=m, hq=z, hs=z)):
        assert norm(lib, **kw) == ALIGN, kw
    over = ctypes.c_void_p(0x100000 + 512)
    assert norm(lib, y_=over) == UNSUPPORTED                      # one row on
    assert norm(lib, y_=x, ldy=512) == UNSUPPORTED                # the same start, another stride


def bwd(lib, dy=x, dt=0, rows=4, cols=256, ld=256, add=None, x_=y, ldx=256, hq=None, hs=None, w=None, wd=0, mean=z, rstd=z,
        center=1, dadd=None, ldadd=256, dx=z, lddx=256, dw=None, db=None, ws=None, n=0):
    return lib.moe_layer_norm_backward(dy, dt, rows, cols, ld, add, x_, ldx, hq, hs, w, wd, mean, rstd, center, dadd, ldadd, dx,
                                       lddx, dw, db, ws, n, None)


def test_norm_backward(lib):
    assert bwd(lib, rows=0, dy=None, x_=None, rstd=None, dx=None) == 0
    for kw in (dict(cols=0), dict(cols=16385), dict(rows=-1), dict(ld=255), dict(ldx=255), dict(lddx=255),
               dict(dadd=y, ldadd=255), dict(dt=3), dict(wd=2), dict(cols=200, x_=None, hq=z, hs=z)):
        assert bwd(lib, **kw) == SHAPE, kw
    for kw in (dict(dy=None), dict(rstd=None), dict(x_=None), dict(hq=y, hs=y), dict(x_=None, hq=y), dict(mean=None),
               dict(dadd=y, dx=None)):
        assert bwd(lib, **kw) == NULL, kw
    for kw in (dict(dy=o), dict(x_=o), dict(dx=o), dict(add=ctypes.c_void_p(0x2)), dict(x_=None, hq=o, hs=y),
               dict(dy=m, x_=None, hq=y, hs=y)):
        assert bwd(lib, **kw) == ALIGN, kw
    over = ctypes.c_void_p(0x100000 + 512)
    assert bwd(lib, dx=over) == UNSUPPORTED                       # over dy, one row on
    assert bwd(lib, add=z, dx=z) == UNSUPPORTED
    assert bwd(lib, x_=None, hq=z, hs=y, dx=z) == UNSUPPORTED
    need = lib.moe_layer_norm_backward_workspace_size(4, 256)
    assert need >= 2 * 256 * 4 and lib.moe_layer_norm_backward_workspace_size(4, 0) == 0
    assert bwd(lib, dw=z) == WORKSPACE
    assert bwd(lib, db=z, ws=y, n=need - 1) == WORKSPACE
    assert bwd(lib, dw=z, ws=m, n=need) == ALIGN


def test_norm_outputs_over_inputs(lib):
    P = lambda v: ctypes.c_void_p(v)
    full = lambda **kw: lib.moe_layer_norm(*[dict(dict(
        x=P(0x100000), dt=0, rows=4, cols=256, ld=256, w=P(0x200000), b=P(0x210000), wd=1, eps=1e-5, c=1, y=P(0x300000), ldy=256,
        m=P(0x400000), r=P(0x410000), yq=P(0x500000), ys=P(0x510000), hq=P(0x600000), hs=P(0x610000), st=None), **kw)[n]
        for n in "x dt rows cols ld w b wd eps c y ldy m r yq ys hq hs st".split()])
    for kw in (dict(yq=P(0x100000)), dict(hq=P(0x100100)), dict(ys=P(0x1007F0)), dict(hs=P(0x100000)), dict(m=P(0x100400)),
               dict(r=P(0x1007FC)), dict(y=P(0x200000)), dict(y=P(0x210000 - 2048 + 16)), dict(m=P(0x200010)), dict(hs=P(0x2103F0))):
        assert full(**kw) == UNSUPPORTED, kw
    for kw in (dict(m=P(0x400002)), dict(r=P(0x410001)), dict(ys=P(0x510002)), dict(hs=P(0x610003))):
        assert full(**kw) == ALIGN, kw
    need = lib.moe_layer_norm_backward_workspace_size(4, 256)
    base = dict(w=P(0x200000), wd=1, mean=P(0x400000), rstd=P(0x410000), dx=P(0x300000), dw=P(0x500000), db=P(0x510000),
                ws=P(0x10000000), n=need, dadd=P(0x620000), add=P(0x630000))
    for kw in (dict(dx=P(0x200010)), dict(dx=P(0x400000)), dict(dx=P(0x410000 - 2048 + 16)), dict(dw=P(0x200000)), dict(db=P(0x410004)),
               dict(dw=x), dict(db=y), dict(dw=P(0x6207FC)), dict(dw=P(0x630FFC)), dict(ws=x), dict(ws=P(0x400000))):
        assert bwd(lib, **dict(base, **kw)) == UNSUPPORTED, kw
    q = dict(x_=None, mean=None, hq=P(0x700000), hs=P(0x710000))
    for kw in (dict(dx=P(0x710000)), dict(dw=P(0x700000)), dict(db=P(0x710000)), dict(ws=P(0x700000))):
        assert bwd(lib, **dict(base, **q, **kw)) == UNSUPPORTED, kw
    for kw in (dict(mean=P(0x400002)), dict(rstd=P(0x410002)), dict(dw=P(0x500001)), dict(db=P(0x510002))):
        assert bwd(lib, **dict(base, **kw)) == ALIGN, kw
    assert bwd(lib, **dict(base, **dict(q, hs=P(0x710002)))) == ALIGN


def test_swiglu_and_ffn_align_fp32_and_maps(lib):
    P = lambda v: ctypes.c_void_p(v)
    base = dict(dh=P(0x2000000), dhs=P(0x2100000), gates=P(0x2200000), sl=P(0x2210000), slots=4, dg=P(0x2220000), ws=P(0x2230000), n=1 << 20,
                off=P(0x2400000), pad=P(0x2410000), t=P(0x2500000), ts=P(0x2600000), c=P(0x2700000), cs=P(0x2800000))
    for name in ("hs", "dhs", "gates", "sl", "dg", "off", "pad", "ts", "cs"):
        assert swi(lib, **dict(base, **{name: P(0x3000002)})) == ALIGN, name
    assert lib.moe_grouped_ffn_fp8_ckpt(x, x, x, 16, 8, 256, 512, x, x, x, x, x, x, P(0x3000002), x, 1 << 30, None, None) == ALIGN


def swi(lib, a=x, hq=y, hs=z, rows=4, F=256, gates=None, sl=None, slots=0, dh=None, dhs=None, dg=None, off=None, pad=None,
        E=1, ld=128, t=None, ts=None, c=None, cs=None, ws=None, n=0):
    return lib.moe_swiglu_backward_ckpt(a, hq, hs, rows, F, gates, sl, slots, dh, dhs, dg, off, pad, E, ld, t, ts, c, cs, ws,
                                        n, None)


def test_swiglu(lib):
    assert swi(lib) == 0                                          # nothing asked for
    assert swi(lib, rows=0, a=None, hq=None, hs=None, dh=x, dhs=x) == 0
    ok = dict(t=x, ts=x, off=z, pad=z)
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(F=0), dict(F=192), dict(slots=-1), dict(slots=1 << 31),
               dict(E=0, **ok), dict(E=1025, **ok), dict(ld=-128, **ok), dict(ld=100, **ok)):
        assert swi(lib, **kw) == SHAPE, kw
    for kw in (dict(dh=x), dict(dhs=x), dict(t=x, off=z, pad=z), dict(cs=x, off=z, pad=z), dict(t=x, ts=x, pad=z),
               dict(c=x, cs=x, off=z), dict(dg=x, slots=4, sl=z), dict(dg=x, slots=4, gates=z), dict(a=None, dh=x, dhs=x),
               dict(hs=None, dh=x, dhs=x)):
        assert swi(lib, **kw) == NULL, kw
    for kw in (dict(a=m, dh=x, dhs=x), dict(hq=m, dh=x, dhs=x), dict(dh=m, dhs=x), dict(t=m, ts=x, off=z, pad=z),
               dict(c=m, cs=x, off=z, pad=z)):
        assert swi(lib, **kw) == ALIGN, kw
    need = lib.moe_swiglu_backward_ckpt_workspace_size(4, 256)
    assert need == 4 * 2 * 4 and lib.moe_swiglu_backward_ckpt_workspace_size(-1, 256) == 0
    g = dict(dg=x, slots=4, gates=z, sl=z)
    assert swi(lib, **g) == WORKSPACE and swi(lib, ws=y, n=need - 1, **g) == WORKSPACE
    assert swi(lib, ws=m, n=need, **g) == ALIGN


def test_ffn_and_combine(lib):
    n4 = [x] * 4
    assert lib.moe_grouped_ffn_fp8_ckpt(None, None, None, 0, 8, 256, 512, *[None] * 4, None, None, None, None, 0, None, None) == 0
    assert lib.moe_grouped_ffn_fp8_ckpt(x, x, x, 16, 8, 256, 512, *n4, x, None, x, x, 1 << 30, None, None) == NULL
    assert lib.moe_grouped_ffn_fp8_ckpt(x, x, x, 16, 8, 256, 512, *n4, x, x, None, x, 1 << 30, None, None) == NULL
    assert lib.moe_grouped_ffn_fp8_ckpt(x, x, x, 16, 8, 256, 512, *n4, x, m, x, x, 1 << 30, None, None) == ALIGN
    assert lib.moe_grouped_ffn_fp8_ckpt(x, x, x, 16, 8, 200, 512, *n4, x, x, x, x, 1 << 30, None, None) == SHAPE
    assert lib.moe_grouped_ffn_fp8_ckpt(x, x, x, 16, 8, 256, 512, *n4, x, x, x, x, 64, None, None) == WORKSPACE
    assert lib.moe_combine_backward(x, x, None, x, 10, 2, 128, 20, x, x, x, None, None) == NULL      # one of the two
    assert lib.moe_combine_backward(x, x, x, x, 10, 2, 128, 20, x, x, None, None, None) == NULL
