"""Pre-activations kept in 8 bits, and the backward from them, on the GPU."""
import pytest
import torch

from tests import ckpt_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def offsets_of(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=torch.int32, device=DEV)


def quant(v):
    b = v.float().unflatten(-1, (-1, 128))
    s = b.abs().amax(-1) / 448.0
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (b / s[..., None]).flatten(-2).to(F8).view(torch.uint8), s


# ------------------------------------------------------------ the forward

@pytest.mark.parametrize("counts,d,F", [([40, 0, 1, 130, 128, 300], 256, 384), ([1], 128, 128), ([0, 517], 512, 128)])
def test_ffn_keeps_h_in_8_bits(L, counts, d, F):
    """out to the bit as without the checkpoint; the codes and scales by their
    rule from the fp32 pre-activations that the other training call writes;
    rows behind the last expert untouched."""
    g = torch.Generator(device=DEV).manual_seed(d + F)
    off, offs = offsets_of(counts)
    A, E, spare = off[-1], len(counts), 9
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    xq, xs = quant(r(A + spare, d) * (0.1 + torch.rand(A + spare, 1, device=DEV, generator=g)))
    w13, w2 = (0.05 * r(E * 2 * F, d)).bfloat16(), (0.05 * r(E * d, F)).bfloat16()
    w13q, w13s = L.fp8_block_quant(w13, 128)
    w2q, w2s = L.fp8_block_quant(w2, 128)
    args = (xq, xs, offs, w13q.view(E, 2 * F, d), w13s.view(E, 2 * F // 128, d // 128), w2q.view(E, d, F),
            w2s.view(E, d // 128, F // 128))
    h = torch.zeros(A + spare, 2 * F, device=DEV)
    ref = L.moe_grouped_ffn_fp8_train(*args, h)
    hq = torch.full((A + spare, 2 * F), 0x55, dtype=torch.uint8, device=DEV)
    hs = torch.full((A + spare, 2 * F // 128), -3.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, q, s = L.moe_grouped_ffn_fp8_ckpt(*args, h_q=hq, h_s=hs, dev_status=st)
    assert L.check_status(st) == 0
    assert torch.equal(out[:A], ref[:A])
    # a tensor as divisor: torch divides by a Python number through its reciprocal
    want_s = h[:A].view(A, -1, 128).abs().amax(2) / torch.full((1, 1), 448.0, device=DEV)
    want_s = torch.where(want_s == 0, torch.ones_like(want_s), want_s)
    assert torch.equal(s[:A], want_s)
    want_q = (h[:A].view(A, -1, 128) * (1.0 / want_s)[..., None]).view(A, -1).to(F8).view(torch.uint8)
    assert torch.equal(q[:A], want_q)
    assert bool((q[A:] == 0x55).all()) and bool((s[A:] == -3.0).all())


def test_ffn_ckpt_empty_and_refusals(L):
    e = lambda *s, dt=torch.uint8: torch.empty(*s, dtype=dt, device=DEV)
    f = torch.float32
    offs = torch.zeros(3, dtype=torch.int32, device=DEV)
    w = (e(2, 512, 256), e(2, 4, 2, dt=f), e(2, 256, 256), e(2, 2, 2, dt=f))
    out, q, s = L.moe_grouped_ffn_fp8_ckpt(e(0, 256), e(0, 2, dt=f), offs, *w)
    assert out.shape == (0, 256) and q.shape == (0, 512) and s.shape == (0, 4)
    with pytest.raises(ValueError):
        L.moe_grouped_ffn_fp8_ckpt(e(8, 256), e(8, 2, dt=f), offs, *w, h_q=e(8, 256))
    with pytest.raises(L.MoEError):
        L.moe_grouped_ffn_fp8_ckpt(e(8, 256), e(8, 2, dt=f), offs, *w, workspace=e(16))


# ----------------------------------------------------------- the backward

def check_codes(q, s, v, e, axis, scale_of):
    """Codes and scales of the values v, known to e."""
    err = (R.decode(q, s, axis) - v).abs()
    assert bool((err <= R.code_error(v, s, axis) + 2 * e).all())
    amax, emax = scale_of(v.abs()), scale_of(e)
    want = torch.where(amax == 0, torch.ones_like(amax), amax / 448)
    assert bool(((s.double() - want).abs() <= 2 * emax / 448 + 2.0 ** -23 * want).all())


def by_row(v):
    return v.view(v.shape[0], -1, 128).amax(2)


def inputs(A, F, g, spread=True):
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)
    h_q, h_s = quant(1.5 * r(A, 2 * F) * (0.2 + 3 * torch.rand(A, 1, device=DEV, generator=g)))
    d_act = (1e-3 * r(A, F) * (torch.rand(A, 1, device=DEV, generator=g) if spread else 1.0)).bfloat16()
    return d_act, h_q, h_s


@pytest.mark.parametrize("rows,F", [(1, 128), (7, 256), (128, 384), (129, 1408), (1000, 128)])
def test_rowwise_and_gates(L, rows, F):
    g = torch.Generator(device=DEV).manual_seed(rows + F)
    d_act, h_q, h_s = inputs(rows, F, g)
    if rows > 4:
        d_act[3] = 0                                                     # a row without a gradient
        h_s[2] = 1e-30                                                   # a row whose pre-activations are next to 0
    slots = rows + 5
    sl2 = torch.full((slots,), -1, dtype=torch.int32, device=DEV)
    at = torch.randperm(slots, device=DEV, generator=g)[:rows]
    sl2[at] = torch.arange(rows, dtype=torch.int32, device=DEV)
    gates = 0.1 + torch.rand(slots, device=DEV, generator=g)
    gates[at[0]] = 0.0                                                   # a gate that is 0
    if slots > 6:
        sl2[(sl2 < 0).nonzero()[0]] = rows + 100                         # a slot that names no row
    dh, dg, _, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, d_gates=True)
    v, act, e, e_act = R.swiglu(d_act, h_q, h_s)
    check_codes(*dh, v, e, 1, by_row)
    ref = torch.zeros(slots, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(ref)
    a = d_act.double()
    ok = (sl2 >= 0) & (sl2 < rows) & (gates != 0)
    rr = sl2[ok].long()
    ref[ok] = (a * act).sum(1)[rr] / gates[ok].double()
    # 3 additions in a lane, 5 over the warp, F / 128 blocks, the products and the quotient; a product
    # below fp32's normal numbers (the row next to 0: 1e-30 squared) is exact to 2^-149 only, three of them an element
    tol[ok] = ((a.abs() * e_act).sum(1) + (12 + F / 128) * R.U * (a * act).abs().sum(1)
               + 3 * F * 2.0 ** -149)[rr] / gates[ok].double()
    assert bool(((dg.double() - ref).abs() <= tol).all())
    assert bool((dg[~ok] == 0).all())
    only = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s)
    assert torch.equal(only[0][0], dh[0]) and torch.equal(only[0][1], dh[1]) and only[1] is None
    alone = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, dh=False, d_gates=True)
    assert alone[0] is None and torch.equal(alone[1], dg)


@pytest.mark.parametrize("counts,F", [([40, 0, 1, 130, 128, 300, 0], 256), ([1], 128), ([0, 127, 129], 384),
                                      ([256] * 3, 128), ([0, 0], 128)])
def test_columnwise(L, counts, F):
    """The weight gradients' operands: zero codes in the padding, nothing behind
    it, spare rows untouched, dh the same bits as alone."""
    g = torch.Generator(device=DEV).manual_seed(F + len(counts))
    off, offs = offsets_of(counts)
    A, spare = off[-1], 11
    rows = A + spare
    d_act, h_q, h_s = inputs(rows, F, g)
    if A > 200:
        d_act[off[3]:off[3] + 128] *= 0                                  # a whole block without a gradient
    pad = L.moe_wgrad_pad_offsets(offs)
    assert pad.tolist() == R.pad_offsets(off)
    P = int(pad[-1])
    ld = P + 256
    new = lambda *s: (torch.full(s, 0x77, dtype=torch.uint8, device=DEV), torch.full((ld // 128, s[0]), -2.0, device=DEV))
    dhT, actT = new(2 * F, ld), new(F, ld)
    gates = 0.1 + torch.rand(rows, device=DEV, generator=g)
    sl2 = torch.arange(rows, dtype=torch.int32, device=DEV)
    sl2[A:] = -1
    dh = (torch.full((rows, 2 * F), 0x33, dtype=torch.uint8, device=DEV), torch.full((rows, 2 * F // 128), -2.0, device=DEV))
    _, dg, _, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, expert_offsets=offs,
                                             pad=pad, ld=ld, dh=dh, d_gates=True, dhT=dhT, actT=actT)
    v, act, e, e_act = R.swiglu(d_act[:A], h_q[:A], h_s[:A])
    by_col = lambda t: t.view(P // 128, 128, -1).amax(1)                 # noqa: E731
    for (q, s), val, err in ((dhT, v, e), (actT, act, e_act)):
        pv, pe = R.padded(val, off, pad.tolist(), P), R.padded(err, off, pad.tolist(), P)
        if P:
            check_codes(q[:, :P].t(), s[:P // 128], pv, pe, 0, by_col)
        live = R.padded(torch.ones(A, 1, dtype=torch.float64, device=DEV), off, pad.tolist(), P)[:, 0] > 0
        assert not bool((q[:, :P][:, ~live] & 0x7F).any())
        assert bool((q[:, P:] == 0x77).all()) and bool((s[P // 128:] == -2.0).all())
    rowwise = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, d_gates=True)
    assert torch.equal(dh[0][:A], rowwise[0][0][:A]) and torch.equal(dh[1][:A], rowwise[0][1][:A])
    assert bool((dh[0][A:] == 0x33).all()) and bool((dh[1][A:] == -2.0).all())
    assert torch.equal(dg, rowwise[1]) and not bool(dg[A:].any())
    for kw in (dict(dhT=True), dict(actT=True)):
        got = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=offs, pad=pad, ld=P, dh=False, **kw)
        one, both = (got[2], dhT) if "dhT" in kw else (got[3], actT)
        assert torch.equal(one[0], both[0][:, :P]) and torch.equal(one[1], both[1][:P // 128])


def test_matches_the_fp32_calls(L):
    """From a checkpoint whose pre-activations fp32 holds exactly, the calls
    that read fp32 give the same dh and operands but for codes at a border."""
    g = torch.Generator(device=DEV).manual_seed(9)
    off, offs = offsets_of([200, 0, 57, 300])
    A, F = off[-1], 384
    d_act, h_q, h_s = inputs(A, F, g)
    h = R.decode(h_q, h_s).float()
    pad = L.moe_wgrad_pad_offsets(offs)
    P = int(pad[-1])
    dh, _, dhT, actT = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=offs, pad=pad, ld=P, dhT=True, actT=True)
    pairs = [(dh, L.moe_swiglu_backward(d_act, h)),
             (dhT, L.moe_wgrad_quant(L.WGRAD_SRC_DH, offs, pad, 2 * F, P, True, h=h, d_act=d_act, F=F)),
             (actT, L.moe_wgrad_quant(L.WGRAD_SRC_ACT, offs, pad, F, P, True, h=h, F=F))]
    for (q, s), (q0, s0) in pairs:
        assert bool(((s - s0).abs() <= 2.0 ** -18 * s0).all())
        assert float((q != q0).float().mean()) < 1e-3


@pytest.mark.parametrize("size", [1e-38, 1e-36, 1e25])
def test_small_and_large_gradients(L, size):
    """Blocks whose scale is subnormal, or large: the codes are as far off as any others."""
    g = torch.Generator(device=DEV).manual_seed(4)
    off, offs = offsets_of([150, 106])
    A, F = off[-1], 128
    d_act, h_q, h_s = inputs(A, F, g, spread=False)
    d_act = (d_act.float() * 1e3 * size).bfloat16()
    pad = L.moe_wgrad_pad_offsets(offs)
    P = int(pad[-1])
    dh, _, dhT, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=offs, pad=pad, ld=P, dhT=True)
    v, _, e, _ = R.swiglu(d_act, h_q, h_s)
    tiny = 2.0 ** -126        # sums and products below the smallest normal keep only its absolute precision
    far = lambda q, s, v, e, axis: (R.decode(q, s, axis) - v).abs() <= (  # noqa: E731
        R.code_error(v, s, axis) * (1 + 2.0 ** -9) + 2 * e + tiny)
    assert bool(far(*dh, v, e, 1).all())
    pv, pe = R.padded(v, off, pad.tolist(), P), R.padded(e, off, pad.tolist(), P)
    assert bool(far(dhT[0].t(), dhT[1], pv, pe, 0).all())


def test_extreme_preactivations(L):
    """Gates far on either side, infinities and NaN of d_act: each stays in its row."""
    A, F = 64, 128
    g = torch.Generator(device=DEV).manual_seed(1)
    d_act, h_q, h_s = inputs(A, F, g)
    h_s[5], h_s[6] = 1.0, 1e4                                            # |gate| up to 448 and 4.5e6
    ref = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s)[0]
    v, _, e, _ = R.swiglu(d_act, h_q, h_s)
    check_codes(*ref, v, e + 1e-30, 1, by_row)
    d_act[9, 4], d_act[11, 100] = float("inf"), float("nan")
    q, s = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s)[0]
    clean = [i for i in range(A) if i not in (9, 11)]
    assert torch.equal(q[clean], ref[0][clean]) and torch.equal(s[clean], ref[1][clean])
    assert bool(s[9].isinf().any()) and bool(q[11].view(F8).float().isnan().any())


def test_bad_maps_stay_inside(L):
    """expert_offsets beyond the rows: nothing outside the buffers is read or written, the rest is right."""
    g = torch.Generator(device=DEV).manual_seed(8)
    A, F = 100, 128
    d_act, h_q, h_s = inputs(A, F, g)
    offs = torch.tensor([0, 60, 180], dtype=torch.int32, device=DEV)     # names 80 rows that are not there
    pad = L.moe_wgrad_pad_offsets(offs)
    P = int(pad[-1])
    dh, _, dhT, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=offs, pad=pad, ld=P, dhT=True)
    good = torch.tensor([0, 60, 100], dtype=torch.int32, device=DEV)
    want = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=good, pad=pad, ld=P, dhT=True)
    assert torch.equal(dh[0], want[0][0])
    assert torch.equal(dhT[0], want[2][0]) and torch.equal(dhT[1], want[2][1])


@pytest.mark.parametrize("ld", [0, 128, 384])
def test_fewer_columns_than_the_maps_name(L, ld):
    """max_pad below pad[E]: every row and gate as without it, the columns of
    the blocks in front of it as with room for all."""
    g = torch.Generator(device=DEV).manual_seed(ld)
    off, offs = offsets_of([40, 0, 130, 257])
    A, F = off[-1], 256
    d_act, h_q, h_s = inputs(A, F, g)
    pad = torch.tensor([0, 128, 128, 384, 768], dtype=torch.int32, device=DEV)
    sl2 = torch.randperm(A, device=DEV, generator=g).int()
    kw = dict(gates=0.1 + torch.rand(A, device=DEV, generator=g), slot_to_sorted=sl2, expert_offsets=offs, pad=pad,
              d_gates=True, dhT=True, actT=True)
    want = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, ld=768, **kw)
    work = torch.full((A * F // 128,), float("nan"), device=DEV)
    got = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, ld=ld, workspace=work, **kw)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1], want[0][1]) and torch.equal(got[1], want[1])
    for a, b in zip(got[2:], want[2:]):
        assert torch.equal(a[0], b[0][:, :ld]) and torch.equal(a[1], b[1][:ld // 128])


def test_empty(L):
    e = lambda *s, dt=torch.uint8: torch.empty(*s, dtype=dt, device=DEV)
    f, i = torch.float32, torch.int32
    offs = torch.zeros(3, dtype=i, device=DEV)
    dh, dg, dhT, actT = L.moe_swiglu_backward_ckpt(
        e(0, 256, dt=torch.bfloat16), e(0, 512), e(0, 4, dt=f), gates=torch.ones(4, 2, device=DEV),
        slot_to_sorted=torch.full((8,), -1, dtype=i, device=DEV), expert_offsets=offs, pad=offs.clone(), ld=128, d_gates=True,
        dhT=True, actT=True)
    assert dh[0].shape == (0, 512) and dg.shape == (4, 2) and not bool(dg.any())


def test_refusals(L):
    g = torch.Generator(device=DEV).manual_seed(8)
    d_act, h_q, h_s = inputs(16, 128, g)
    with pytest.raises(ValueError):
        L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, d_gates=True)
    with pytest.raises(ValueError):
        L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, dhT=True, ld=128)
    with pytest.raises(ValueError):
        L.moe_swiglu_backward_ckpt(d_act, h_q[:, :128].contiguous(), h_s)
    with pytest.raises(TypeError):
        L.moe_swiglu_backward_ckpt(d_act.float(), h_q, h_s)
    with pytest.raises(L.MoEError):
        L.moe_swiglu_backward_ckpt(d_act[:, :96].contiguous(), h_q[:, :192].contiguous(), h_s[:, :1].contiguous())
    offs = torch.tensor([0, 16], dtype=torch.int32, device=DEV)
    with pytest.raises(L.MoEError):
        L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, expert_offsets=offs, pad=offs * 8, ld=100, actT=True)
    with pytest.raises(L.MoEError):
        L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=torch.ones(16, device=DEV),
                                   slot_to_sorted=torch.arange(16, dtype=torch.int32, device=DEV), d_gates=True,
                                   workspace=torch.empty(8, dtype=torch.uint8, device=DEV))


def test_streams_and_graph(L):
    g = torch.Generator(device=DEV).manual_seed(6)
    off, offs = offsets_of([300, 0, 212])
    A, F = off[-1], 256
    d_act, h_q, h_s = inputs(A, F, g)
    other = inputs(A, F, g)
    pad = L.moe_wgrad_pad_offsets(offs)
    P = int(pad[-1])
    gates, sl2 = torch.rand(A, device=DEV, generator=g) + 0.1, torch.randperm(A, device=DEV, generator=g).int()

    def run(stream=None):
        dh, dg, dhT, actT = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, expert_offsets=offs,
                                                       pad=pad, ld=P, d_gates=True, dhT=True, actT=True, stream=stream)
        return (*dh, dg, *dhT, *actT)

    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for t, o in zip((d_act, h_q, h_s), other):
        t.copy_(o)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip([t.clone() for t in held], run()))


@pytest.mark.parametrize("T,k,d", [(5, 2, 128), (300, 3, 2048), (40, 2, 8320)])
def test_combine_backward_without_outputs(L, T, k, d):
    """The rows to the bit as with the experts' outputs given."""
    g = torch.Generator(device=DEV).manual_seed(d)
    A = T * k
    dy = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    gates = torch.rand(T, k, device=DEV, generator=g)
    sl2 = torch.randperm(A, device=DEV, generator=g).int()
    sl2[1] = -1
    out = torch.randn(A, d, device=DEV, generator=g).bfloat16()
    mk = lambda: (torch.full((A, d), 0x11, dtype=torch.uint8, device=DEV), torch.full((A, d // 128), -1.0, device=DEV))
    a, b = mk(), mk()
    L.moe_combine_backward(dy, gates, out, sl2, *a)
    q, s, dg = L.moe_combine_backward(dy, gates, None, sl2, *b)
    assert dg is None and torch.equal(a[0], q) and torch.equal(a[1], s)
    with pytest.raises(ValueError):
        L.moe_combine_backward(dy, gates, None, sl2, d_gates=torch.empty(T, k, device=DEV))
