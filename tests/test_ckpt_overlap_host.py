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
