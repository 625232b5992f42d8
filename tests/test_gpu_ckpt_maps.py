"""The SwiGLU backward from 8 bits with maps that name rows that are not there
or leave rows out: every buffer lies inside a larger one, whose rows on either
side stay as they were and do not show in the results."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 256               # rows on either side: more than a block's 128


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def inner(rows, shape, dtype, fill):
    """[rows, *shape] within `GUARD` rows more on either side, all of `fill` -> the whole, the inner part."""
    whole = torch.full((rows + 2 * GUARD, *shape), fill, dtype=dtype, device=DEV)
    return whole, whole[GUARD:GUARD + rows]


def named(off, pad, E, rows, ld):
    """(padded column, row) of every row that a whole block of the maps holds, by the header's rules."""
    got = []
    for kb in range(max(0, min(pad[E], ld)) // 128):
        for e in range(E):
            if not pad[e] <= 128 * kb < pad[e + 1]:
                continue
            r0 = off[e] + 128 * kb - pad[e]
            if r0 >= 0:
                got += [(128 * kb + i, r0 + i) for i in range(128) if r0 + i < min(rows, off[e + 1])]
    return got


MAPS = [([-5, 60], [0, 128]),                  # rows in front of the first
        ([-200, 100], [0, 384]),               # a whole block in front of it, and one across it
        ([0, 60], [128, 256]),                 # a first column behind 0
        ([70, 100], [128, 256]),               # the same with rows in front of the first expert's
        ([0, 40, 100], [256, 384, 512]),
        ([0, 60, 180], [0, 128, 256]),         # rows behind the last
        ([0, -300, 90], [0, 128, 640])]        # an expert that starts in front of its own end


@pytest.mark.parametrize("off,pad", MAPS)
def test_rows_outside_are_left_alone(L, off, pad):
    A, F, E = 100, 128, len(off) - 1
    g = torch.Generator(device=DEV).manual_seed(len(off) + pad[-1])
    ld = pad[-1] + 128
    bf, u8, f32 = torch.bfloat16, torch.uint8, torch.float32
    # in front of and behind the rows: NaN codes and NaN, which would show in any code or scale formed from them
    _, d_act = inner(A, (F,), bf, float("nan"))
    _, h_q = inner(A, (2 * F,), u8, 0x7F)
    _, h_s = inner(A, (2 * F // 128,), f32, float("nan"))
    d_act.copy_(1e-3 * torch.randn(A, F, device=DEV, generator=g))
    h_q.copy_(torch.randint(0, 0x70, (A, 2 * F), device=DEV, generator=g))
    h_s.copy_(0.01 * torch.rand(A, 2 * F // 128, device=DEV, generator=g))
    outs = [inner(A, (2 * F,), u8, 0x55), inner(A, (2 * F // 128,), f32, -3.0),
            inner(2 * F, (ld,), u8, 0x55), inner(ld // 128, (2 * F,), f32, -3.0),
            inner(F, (ld,), u8, 0x55), inner(ld // 128, (F,), f32, -3.0), inner(A, (F // 128,), f32, -3.0)]
    (_, dq), (_, ds), (_, tq), (_, ts), (_, aq), (_, as_), (_, work) = outs
    gates = 0.1 + torch.rand(A, device=DEV, generator=g)
    sl2 = torch.randperm(A, device=DEV, generator=g).int()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    want_dh = L.moe_swiglu_backward_ckpt(d_act.clone(), h_q.clone(), h_s.clone())[0]
    _, dg, _, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, expert_offsets=i32(off),
                                             pad=i32(pad), ld=ld, dh=(dq, ds), d_gates=True, dhT=(tq, ts), actT=(aq, as_),
                                             workspace=work)
    torch.cuda.synchronize()
    for whole, part in outs:
        fill = whole[0].clone()
        assert bool((whole[:GUARD] == fill).all()) and bool((whole[GUARD + part.shape[0]:] == fill).all())
    where = named(off, pad, E, A, ld)
    rows = torch.zeros(A, dtype=torch.bool)
    rows[[r for _, r in where]] = True
    rows = rows.to(DEV)
    assert torch.equal(dq[rows], want_dh[0][rows]) and torch.equal(ds[rows], want_dh[1][rows])
    assert bool((dq[~rows] == 0x55).all()) and bool((ds[~rows] == -3.0).all())
    # the columns: codes of the rows that are there, zeros for the others, nothing of what lies around
    P = pad[E]
    live = torch.zeros(P, dtype=torch.bool, device=DEV)
    live[[c for c, _ in where]] = True
    for q, s in ((tq, ts), (aq, as_)):
        assert not bool((q[:, :P][:, ~live] & 0x7F).any()) and bool((q[:, P:] == 0x55).all())
        assert bool(((q[:, :P] & 0x7F) != 0x7F).all()) and bool(s[:P // 128].isfinite().all())
        assert bool((s[:P // 128] > 0).all()) and bool((s[P // 128:] == -3.0).all())
    r = sl2.long()
    dot_rows = rows[r]
    assert bool(dg[dot_rows].isfinite().all())


LEFT_OUT = [([10, 60], [0, 128]),               # rows in front of the first expert's
            ([0, 60, 300], [0, 128, 128]),      # an expert without columns
            ([0, 60, 300], [0, 128, 256]),      # one with fewer columns than rows
            ([0, 60, 300], [128, 256, 512]),    # columns that begin behind 0
            ([0, 60, 300], [256, 0, 384]),      # columns out of order
            ([0, 300, 60], [0, 384, 512]),      # rows out of order
            ([0, 60, 300], [0, 128, 0])]        # no columns at all


@pytest.mark.parametrize("off,pad", MAPS + LEFT_OUT)
def test_gates_of_rows_left_out(L, off, pad):
    """A slot whose row no block of the maps holds has a gradient of 0, whatever
    the workspace held; the others as without maps.  (Maps out of order may leave
    out more rows: each slot has the one or the other.)"""
    A, F, E = 300, 256, len(off) - 1
    g = torch.Generator(device=DEV).manual_seed(pad[-1] + off[-1])
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    d_act, h_s = (1e-3 * r(A, F)).bfloat16(), 0.01 + 0.01 * torch.rand(A, 2 * F // 128, device=DEV, generator=g)
    h_q = torch.randint(0, 0x70, (A, 2 * F), device=DEV, generator=g, dtype=torch.uint8)
    gates, sl2 = 0.1 + torch.rand(A, device=DEV, generator=g), torch.randperm(A, device=DEV, generator=g).int()
    want = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, dh=False, d_gates=True)[1]
    assert bool((want != 0).all())
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    ld = 512
    work = torch.full((A * F // 128,), float("nan"), device=DEV)
    _, dg, _, _ = L.moe_swiglu_backward_ckpt(d_act, h_q, h_s, gates=gates, slot_to_sorted=sl2, expert_offsets=i32(off),
                                             pad=i32(pad), ld=ld, d_gates=True, dhT=True, actT=True, workspace=work)
    rows = torch.zeros(A, dtype=torch.bool)
    rows[[row for _, row in named(off, pad, E, A, max(pad))]] = True
    has = rows.to(DEV)[sl2.long()]
    if off == sorted(off) and pad == sorted(pad):
        assert torch.equal(dg, torch.where(has, want, torch.zeros_like(want)))
    else:
        assert bool(((dg == 0) | (dg == want)).all())
