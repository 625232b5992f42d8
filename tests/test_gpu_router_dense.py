"""The router over all experts (dense logits, balance and z losses with counts
and gradients, the dense backward) against 64-bit forms.

Tolerances.  Products: every fp32 addition is off by at most 2^-23 of the
partial sum (a tensor-core sum may truncate), a sum of K products has at most
K / 2 + 32 of them in a row (16 products enter each, in up to three parts), so
an entry is off by at most (K + 64) 2^-24 sum |a||b|; the roundings are
independent, so the norm of all errors is held to (8 + 2 sqrt(K)) 2^-24 of the
norm of the result.  Balance: an exponential is good to 2^-23 and its argument
to 2^-24 R (R the row's range), a sum of E terms to (E / 32 + 6) 2^-24, and six
operations follow: rel = 2^-24 (24 + 2 min(R, 110) + E / 16), on the sum of the
absolute parts of an entry."""
import numpy as np
import pytest
import torch

from tests import loss_refs as R

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = 0, 1


@pytest.fixture(scope="module")
def L():
    from block_scaled_fp8_router_gb300 import moe_r3
    return moe_r3


def _xw(T, d, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    w = (0.05 * torch.randn(E, d, device="cuda", generator=g)).bfloat16()
    return x, w, g


def _product(got, a, b, what):
    """got = a @ b, a and b 64-bit."""
    K = a.shape[1]
    want, size = a @ b, a.abs() @ b.abs()
    err = (got.double() - want).abs()
    assert bool((err <= (K + 64) * 2.0 ** -24 * size + 2.0 ** -126).all()), (what, float((err / size.clamp_min(1e-300)).max()))
    if want.numel():
        assert float(err.norm()) <= (8 + 2 * K ** 0.5) * 2.0 ** -24 * float(want.norm()) + 1e-38, \
            (what, float(err.norm() / want.norm()))


SHAPES = [(1, 128, 1), (3, 128, 8), (127, 256, 37), (128, 384, 64), (129, 128, 128), (300, 2048, 64), (257, 7168, 256),
          (1000, 512, 300), (64, 256, 1024), (2500, 640, 160), (4093, 1408, 64), (700, 256, 513)]


@pytest.mark.parametrize("T,d,E", SHAPES)
def test_router_logits(L, T, d, E):
    x, w, _ = _xw(T, d, E, T + d + E)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    l = L.moe_router_logits(x, w, dev_status=st)
    assert int(st) == 0
    _product(l, x.double(), w.double().t(), "logits")
    assert torch.equal(l, L.moe_router_logits(x, w))                           # the same bits again


def test_router_logits_agree_with_the_router(L):
    """Within rounding of the routing kernel's fma chain."""
    x, w, _ = _xw(513, 1024, 96, 5)
    chain = torch.empty(513, 96, device="cuda")
    L.moe_route_topk(x, w, 4, SOFTMAX, logits_out=chain)
    size = x.double().abs() @ w.double().abs().t()
    assert bool(((L.moe_router_logits(x, w).double() - chain.double()).abs() <= 2 * (1024 + 64) * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("T,d,E", SHAPES)
def test_router_backward_dense(L, T, d, E):
    x, w, g = _xw(T, d, E, T + d + E + 1)
    dl = torch.randn(T, E, device="cuda", generator=g) * torch.exp(2 * torch.randn(T, 1, device="cuda", generator=g))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dx, dw = L.moe_router_backward_dense(x, w, dl, dev_status=st)
    assert int(st) == 0
    _product(dx, dl.double(), w.double(), "dx")
    _product(dw, dl.double().t(), x.double(), "dw")
    dx1, none = L.moe_router_backward_dense(x, w, dl, dw_router=False)
    assert none is None and torch.equal(dx, dx1)
    none, dw1 = L.moe_router_backward_dense(x, w, dl, dx=False)
    assert none is None and torch.equal(dw, dw1)


def test_router_backward_dense_keeps_24_bits(L):
    """Entries whose low bits matter: d_logits with full mantissas against
    one-hot weights come back to within the last bit, zeros as zeros, and
    infinities and NaN stay in their row (dx) and column (dW_r)."""
    T, d, E = 200, 256, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    dl = torch.randn(T, E, device="cuda", generator=g) * torch.exp2(torch.randint(-90, 90, (T, E), device="cuda", generator=g).float())
    w = torch.zeros(E, d, device="cuda", dtype=torch.bfloat16)
    w[torch.arange(E), torch.arange(E)] = 1
    x = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    x[torch.arange(T), torch.arange(T)] = 1
    dx, dw = L.moe_router_backward_dense(x, w, dl)
    assert bool(((dx[:, :E] - dl).abs() <= 2.0 ** -23 * dl.abs()).all()) and dx[:, E:].eq(0).all()
    assert bool(((dw[:, :T] - dl.t()).abs() <= 2.0 ** -23 * dl.t().abs()).all()) and dw[:, T:].eq(0).all()
    dl[7, 3] = float("nan")
    dl[9, 5] = float("inf")
    w[:], x[:] = 1, 1
    dx, dw = L.moe_router_backward_dense(x, w, dl)
    assert not torch.isfinite(dx[7]).any() and not torch.isfinite(dx[9]).any()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[[7, 9]] = False
    assert torch.isfinite(dx[rest]).all()
    assert not torch.isfinite(dw[3]).any() and not torch.isfinite(dw[5]).any()


@pytest.mark.parametrize("T,d,E", [(200, 256, 64), (1500, 512, 256), (4000, 7168, 256)])
def test_router_backward_dense_infinities(L, T, d, E):
    """Infinite and NaN gradients give what the fp32 product gives: the sign of
    the infinity, NaN where two meet, a NaN of any payload."""
    g = torch.Generator(device="cuda").manual_seed(T)
    dl = torch.randn(T, E, device="cuda", generator=g)
    inf = float("inf")
    dl[9, 5], dl[20, 2], dl[30, 1], dl[30, 2] = inf, -inf, inf, -inf
    dl.view(torch.int32)[7, 3] = 0x7F800001
    x = torch.ones(T, d, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(E, d, device="cuda", dtype=torch.bfloat16)
    w[:, 1::2] = -1
    dx, dw = L.moe_router_backward_dense(x, w, dl)
    sign = w[0].float()
    assert torch.equal(dx[9], inf * sign) and torch.equal(dx[20], -inf * sign)
    assert dx[30].isnan().all() and dx[7].isnan().all()
    assert dw[5].eq(inf).all() and dw[1].eq(inf).all() and dw[2].eq(-inf).all() and dw[3].isnan().all()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[[7, 9, 20, 30]] = False
    cols = torch.ones(E, dtype=torch.bool, device="cuda")
    cols[[1, 2, 3, 5]] = False
    assert dx[rest].isfinite().all() and dw[cols].isfinite().all()


def test_dense_empty(L):
    x, w, _ = _xw(0, 128, 8, 1)
    assert L.moe_router_logits(x, w).shape == (0, 8)
    dx, dw = L.moe_router_backward_dense(x, w, torch.empty(0, 8, device="cuda"))
    assert dx.shape == (0, 128) and dw.eq(0).all()
    losses, counts, d = L.moe_balance_loss(torch.empty(0, 8, device="cuda"),
                                           torch.empty(0, 2, dtype=torch.int32, device="cuda"), SOFTMAX, 0.1)
    assert losses.eq(0).all() and counts.eq(0).all() and d.shape == (0, 8)


# ------------------------------------------------------------ balance loss

def _bal(T, E, k, seed, seqs=1, mask=False, gates=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = 2 * torch.randn(T, E, device="cuda", generator=g) + torch.randn(E, device="cuda", generator=g)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, 1).indices.int()
    m = torch.rand(T, device="cuda", generator=g) < 0.7 if mask else None
    off = None
    if seqs > 1:
        cut = torch.randint(0, T + 1, (seqs - 1,), device="cuda", generator=g).sort().values
        off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).int()
    dg = 1e-2 * torch.randn(T, k, device="cuda", generator=g) if gates else None
    return l, ids, m, off, dg


def _check_balance(L, l, ids, m, off, dg, score, renorm=1, alpha=0.1, zeta=0.01, scale=1.0, gs=1.0):
    T, E = l.shape
    losses, counts, d = L.moe_balance_loss(l, ids, score, alpha, z_coef=zeta, token_mask=m, seq_offsets=off,
                                           d_gates=dg, renorm=renorm, route_scale=scale, grad_scale=gs)
    wl, wc, wd = R.balance(l, ids, score, alpha, zeta, m, off, dg, renorm, scale, gs)
    assert torch.equal(counts.long(), wc)
    span = float((l.amax(1) - l.amin(1)).max())
    rel = 2.0 ** -24 * (24 + 2 * min(span, 110) + E / 16)
    assert bool(((losses.double() - wl).abs() <= 4 * rel * wl.abs() + 1e-30).all()), (losses, wl)
    # the parts of an entry: q (f + sum f q), 2 lse p, and the gates' dg (its largest in the row bounds them)
    s = torch.softmax(l.double(), 1) if score == SOFTMAX else torch.sigmoid(l.double())
    q = s / s.sum(1, keepdim=True)
    n = float(T if m is None else m.sum())
    fmax = float((wc.double() * E).max()) if wc.numel() else 0.0
    lse = torch.logsumexp(l.double(), 1, keepdim=True).abs()
    nb = wc.sum(1).clamp_min(1).double() / ids.shape[1]
    fb = float((wc.double().amax(1) * E / (ids.shape[1] * nb) / nb).max())
    size = gs * alpha * fb * 2 * q + gs * 2 * zeta * (lse + 1) / max(n, 1) * torch.softmax(l.double(), 1)
    if dg is not None:
        part = scale * dg.double().abs().sum(1, keepdim=True)
        if renorm == 0 and score == SOFTMAX:
            size = size + part * q
        size = size.scatter_add(1, ids.long(), 2 * part.expand(-1, ids.shape[1]))
    err = (d.double() - wd).abs()
    assert bool((err <= 4 * rel * size + 1e-35).all()), float((err / size).max() / rel)
    return losses, counts, d


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,k,seqs,mask,gates,renorm", [
    (1, 1, 1, 1, False, False, 1), (1, 8, 2, 1, False, True, 1), (7, 8, 8, 3, False, True, 0), (256, 8, 2, 1, False, False, 1),
    (333, 37, 4, 5, True, True, 1), (333, 37, 4, 5, True, True, 0), (1000, 64, 6, 1, True, True, 1),
    (513, 256, 8, 7, False, True, 1), (513, 256, 8, 1, False, True, 0), (300, 1024, 32, 40, True, True, 1),
    (2049, 160, 8, 2, False, False, 1), (5000, 300, 3, 600, True, False, 1), (700, 512, 4, 1, False, True, 1)])
def test_balance(L, score, T, E, k, seqs, mask, gates, renorm):
    a = _bal(T, E, k, T + E + k, seqs, mask, gates)
    one = _check_balance(L, *a, score, renorm=renorm, scale=2.5, gs=3.0)
    two = _check_balance(L, *a, score, renorm=renorm, scale=2.5, gs=3.0)
    for u, v in zip(one, two):                                                 # the same bits again
        assert torch.equal(u, v)


def test_balance_without_gradient_or_z(L):
    l, ids, m, off, _ = _bal(400, 64, 4, 2, 3, True)
    a = L.moe_balance_loss(l, ids, SIGMOID, 0.1, token_mask=m, seq_offsets=off)
    b = L.moe_balance_loss(l, ids, SIGMOID, 0.1, token_mask=m.to(torch.uint8), seq_offsets=off, d_logits=False)
    assert b[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and a[0][1] == 0


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_balance_masked_tokens_hold_anything(L, score):
    """Uncounted tokens: NaN and infinite logits without gates' gradients give
    zero rows and change nothing; all of them uncounted gives zeros."""
    l, ids, m, off, dg = _bal(300, 64, 4, 11, 4, True, True)
    dg[~m] = 0
    a = L.moe_balance_loss(l, ids, score, 0.1, z_coef=0.01, token_mask=m, seq_offsets=off, d_gates=dg)
    l2 = l.clone()
    l2[~m] = float("nan")
    l2[torch.nonzero(~m)[0, 0]] = float("-inf")
    l2[torch.nonzero(~m)[1, 0]] = float("inf")
    b = L.moe_balance_loss(l2, ids, score, 0.1, z_coef=0.01, token_mask=m, seq_offsets=off, d_gates=dg)
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    assert b[2][~m].eq(0).all()
    c = L.moe_balance_loss(l2, ids, score, 0.1, z_coef=0.01, token_mask=torch.zeros_like(m), seq_offsets=off)
    assert c[0].eq(0).all() and c[1].eq(0).all() and c[2].eq(0).all()


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_balance_masked_experts(L, score):
    """Experts at -inf and at the lowest fp32: no probability, no gradient; a
    token with every expert at -inf adds nothing."""
    l, ids, m, off, _ = _bal(200, 40, 3, 12)
    l[:, 10:20] = float("-inf")
    l[:, 20:25] = torch.finfo(torch.float32).min
    losses, counts, d = L.moe_balance_loss(l, ids, score, 0.1, z_coef=0.01)
    wl, wc, wd = R.balance(l, ids, score, 0.1, 0.01)
    assert torch.equal(counts.long(), wc)
    assert bool(((losses.double() - wl).abs() <= 2.0 ** -18 * wl).all())
    assert d[:, 10:25].eq(0).all() and torch.isfinite(d).all()
    assert float((d.double() - wd.nan_to_num(0)).norm()) <= 2.0 ** -18 * float(wd.nan_to_num(0).norm())
    l[5] = float("-inf")
    losses, counts, d = L.moe_balance_loss(l, ids, score, 0.1, z_coef=0.01)
    assert torch.equal(counts.long(), wc) and torch.isfinite(losses).all() and d[5].eq(0).all()


def test_balance_bad_ids_and_offsets(L):
    """Ids outside [0, E) are not counted, offsets outside [0, T] or decreasing
    are flagged; nothing is read or written out of range."""
    l, ids, m, off, dg = _bal(100, 16, 2, 13, 3, False, True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.moe_balance_loss(l, ids, SIGMOID, 0.1, seq_offsets=off, d_gates=dg, dev_status=st)
    assert int(st) == 0
    bad = ids.clone()
    bad[3, 0], bad[4, 1], bad[5, 1] = -1, 16, bad[5, 0]
    losses, counts, d = L.moe_balance_loss(l, bad, SIGMOID, 0.1, seq_offsets=off, d_gates=dg, dev_status=st)
    assert int(st) == L.MOE_DEV_BAD_IDS
    assert int(counts.sum()) == 100 * 2 - 2 and torch.isfinite(d).all()
    zero = dg.clone()
    zero[3:6] = 0
    rest = L.moe_balance_loss(l, bad, SIGMOID, 0.1, seq_offsets=off, d_gates=zero)[2]
    assert torch.equal(rest, d)                       # no gradient through a bad token's gates
    for o in ([0, 50, 40, 100], [-5, 10, 20, 100], [0, 10, 20, 500]):
        st.zero_()
        losses, counts, d = L.moe_balance_loss(l, ids, SIGMOID, 0.1, dev_status=st,
                                               seq_offsets=torch.tensor(o, dtype=torch.int32, device="cuda"))
        assert int(st) == L.MOE_DEV_ROWS
        assert int(counts.sum()) <= 200 and torch.isfinite(d).all()


def test_balance_gradient_against_differences(L):
    """Central differences of the 64-bit losses and gates (step 1e-4: 1e-8 of the entries)."""
    l, ids, m, off, dg = _bal(12, 10, 3, 14, 2, True, True)
    for score, renorm in ((SOFTMAX, 0), (SOFTMAX, 1), (SIGMOID, 0), (SIGMOID, 1)):
        d = L.moe_balance_loss(l, ids, score, 0.5, z_coef=0.3, token_mask=m, seq_offsets=off, d_gates=dg,
                               renorm=renorm, route_scale=1.5)[2]

        def f(z):
            s = R.balance(z, ids, score, 0.5, 0.3, m, off)[0].sum()
            return float(s + (R.gates(z, ids.long(), score, renorm, 1.5) * dg.double()).sum())
        for t, e in [(0, 0), (3, int(ids[3, 1])), (7, 9), (11, int(ids[11, 0]))]:
            up, dn = l.double(), l.double()
            up[t, e] += 1e-4
            dn[t, e] -= 1e-4
            num = (f(up) - f(dn)) / 2e-4
            assert abs(num - float(d[t, e])) < 1e-6 * max(1.0, abs(num)), (score, renorm, t, e, num, float(d[t, e]))


def test_dense_router_follows_the_stream_and_graphs(L):
    x, w, g = _xw(300, 512, 64, 31)
    l0, ids, m, off, dg = _bal(300, 64, 4, 32, 3, True, True)
    l = L.moe_router_logits(x, w)
    lo, co, dl = L.moe_balance_loss(l, ids, SIGMOID, 0.1, z_coef=0.01, token_mask=m, seq_offsets=off, d_gates=dg)
    dx, dw = L.moe_router_backward_dense(x, w, dl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    u8 = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    w1, w2, w3 = (u8(L.moe_router_logits_workspace_size(300, 512, 64)), u8(L.moe_balance_loss_workspace_size(300, 64, 3)),
                  u8(L.moe_router_backward_dense_workspace_size(300, 512, 64)))
    with torch.cuda.stream(side):
        z = x * 1.0
        b = L.moe_router_logits(z, w, workspace=w1)
        b = L.moe_balance_loss(b, ids, SIGMOID, 0.1, z_coef=0.01, token_mask=m, seq_offsets=off, d_gates=dg, workspace=w2)
        c = L.moe_router_backward_dense(z, w, b[2], workspace=w3)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(b[0], lo) and torch.equal(b[1], co) and torch.equal(b[2], dl)
    assert torch.equal(c[0], dx) and torch.equal(c[1], dw)
    z = torch.zeros_like(x)
    out = dict(l=torch.empty_like(l), lo=torch.empty_like(lo), co=torch.empty_like(co), dl=torch.empty_like(dl),
               dx=torch.empty_like(dx), dw=torch.empty_like(dw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.moe_router_logits(z, w, logits=out["l"], workspace=w1)
        L.moe_balance_loss(out["l"], ids, SIGMOID, 0.1, z_coef=0.01, token_mask=m, seq_offsets=off, d_gates=dg,
                           counts=out["co"], losses=out["lo"], d_logits=out["dl"], workspace=w2)
        L.moe_router_backward_dense(z, w, out["dl"], dx=out["dx"], dw_router=out["dw"], workspace=w3)
    for _ in range(2):
        z.copy_(x)
        for t in (w1, w2, w3):
            t.fill_(0xFF)                              # a workspace's contents do not matter
        graph.replay()
        assert torch.equal(out["l"], l) and torch.equal(out["lo"], lo) and torch.equal(out["co"], co)
        assert torch.equal(out["dl"], dl) and torch.equal(out["dx"], dx) and torch.equal(out["dw"], dw)


@pytest.mark.slow
def test_balance_many_tokens(L):
    """T * E beyond 2^31 logits' bytes (token offsets past 32 bits)."""
    T, E, k = 9_000_000, 256, 2
    l = torch.empty(T, E, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    ids = torch.stack([torch.arange(T, device="cuda") % E, (torch.arange(T, device="cuda") + 7) % E], 1).int()
    losses, counts, d = L.moe_balance_loss(l, ids, SOFTMAX, 0.1)
    want = torch.bincount(ids.long().reshape(-1), minlength=E)
    assert torch.equal(counts[0].long(), want)
    q = torch.softmax(l[-5:].double(), 1)
    f = want.double() * E / (k * T)
    ref = 0.1 / T * q * (f - (q * f).sum(1, keepdim=True))
    assert float((d[-5:].double() - ref).abs().max()) <= 2.0 ** -18 * float((0.2 / T * q).abs().max())
