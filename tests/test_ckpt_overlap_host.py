"""The 8-bit calls refuse outputs and workspaces over an input or over one
another on the host, before anything is launched (fake pointers, no GPU)."""
import ctypes

import pytest

UNSUPPORTED = 6
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3._lib


def one_over_another(call, spans, outs):
    """Every output's first bytes laid over the last 16 of every other buffer, and its last 16 over the other's first."""
    base = {n: 0x10000000 * (i + 1) for i, n in enumerate(spans)}
    for o in outs:
        for n in spans:
            if n == o:
                continue
            for at in (base[n] + max(0, spans[n] - 16) // 256 * 256, base[n] - max(0, spans[o] - 16) // 256 * 256):
                assert at + spans[o] > base[n] and base[n] + spans[n] > at
                assert call(**{m: P(at if m == o else v) for m, v in base.items()}) == UNSUPPORTED, (o, n, hex(at - base[n]))


def test_swiglu(lib):
    rows, F, E, ld, slots = 300, 256, 4, 640, 310
    spans = dict(a=rows * F * 2, hq=rows * 2 * F, hs=rows * 2 * F // 128 * 4, gates=slots * 4, sl=slots * 4, dh=rows * 2 * F,
                 dhs=rows * 2 * F // 128 * 4, dg=slots * 4, off=(E + 1) * 4, pad=(E + 1) * 4, t=2 * F * ld,
                 ts=ld // 128 * 2 * F * 4, c=F * ld, cs=ld // 128 * F * 4, ws=rows * F // 128 * 4)

    def call(a, hq, hs, gates, sl, dh, dhs, dg, off, pad, t, ts, c, cs, ws):
        return lib.moe_swiglu_backward_ckpt(a, hq, hs, rows, F, gates, sl, slots, dh, dhs, dg, off, pad, E, ld, t, ts, c, cs,
                                            ws, spans["ws"], None)

    one_over_another(call, spans, ["dh", "dhs", "dg", "t", "ts", "c", "cs", "ws"])


def test_ffn(lib):
    rows, E, d, F = 300, 4, 256, 384
    n = lib.moe_grouped_ffn_workspace_size(rows, d, F)
    spans = dict(x=rows * d, xs=rows * d // 128 * 4, off=(E + 1) * 4, w13=2 * E * F * d, w13s=2 * E * F * d // 16384 * 4,
                 w2=E * F * d, w2s=E * F * d // 16384 * 4, out=rows * d * 2, hq=rows * 2 * F, hs=rows * 2 * F // 128 * 4, ws=n)

    def call(x, xs, off, w13, w13s, w2, w2s, out, hq, hs, ws):
        return lib.moe_grouped_ffn_fp8_ckpt(x, xs, off, rows, E, d, F, w13, w13s, w2, w2s, out, hq, hs, ws, n, None, None)

    one_over_another(call, spans, ["out", "hq", "hs", "ws"])


def test_norm(lib):
    rows, cols = 300, 256
    n = rows * cols
    spans = dict(x=2 * n, w=4 * cols, b=4 * cols, y=2 * n, mean=4 * rows, rstd=4 * rows, yq=n, ys=n // 32, hq=n, hs=n // 32)

    def call(x, w, b, y, mean, rstd, yq, ys, hq, hs):
        return lib.moe_layer_norm(x, 0, rows, cols, cols, w, b, 1, 1e-5, 1, y, cols, mean, rstd, yq, ys, hq, hs, None)

    # y over x is the caller's to ask for, row on row
    one_over_another(call, spans, ["mean", "rstd", "yq", "ys", "hq", "hs"])


@pytest.mark.parametrize("codes", [False, True])
def test_norm_backward(lib, codes):
    rows, cols = 300, 256
    n, ws = rows * cols, lib.moe_layer_norm_backward_workspace_size(rows, cols)
    spans = dict(dy=2 * n, dya=4 * n, w=4 * cols, rstd=4 * rows, dxa=2 * n, dx=2 * n, dw=4 * cols, db=4 * cols, ws=ws)
    spans.update(dict(hq=n, hs=n // 32) if codes else dict(x=2 * n, mean=4 * rows))

    def call(dy, dya, w, rstd, dxa, dx, dw, db, ws, x=None, mean=None, hq=None, hs=None):
        return lib.moe_layer_norm_backward(dy, 0, rows, cols, cols, dya, x, cols, hq, hs, w, 1, mean, rstd, 1, dxa, cols, dx,
                                           cols, dw, db, ws, spans["ws"], None)

    one_over_another(call, spans, ["dw", "db", "ws"])
