"""64-bit forms of the norm, of the SwiGLU backward from 8-bit pre-activations
and of the E4M3 block codes, for the tests (torch on the CPU or GPU; no code
of the library or of the oracle)."""
import torch

U = 2.0 ** -24            # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def decode(q, s, axis=1):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, axis)


def code_error(v, s, axis=1):
    """How far E4M3 codes at scale s may be from the values v: half a step (of
    v's binade, or of the subnormals), and the scale's and the reciprocal's
    own roundings of the quotient."""
    return v.abs() * (2.0 ** -4 + 2.0 ** -21) + s.double().repeat_interleave(128, axis) * 2.0 ** -10


def norm(x, w, b, eps, center):
    x = x.double()
    mu = x.mean(1, keepdim=True) if center else torch.zeros_like(x[:, :1])
    r = 1.0 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + eps)
    h = (x - mu) * r
    y = h * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return y, mu[:, 0], r[:, 0], h


def norm_backward(dy, h, r, w, center, dy_add=None, dx_add=None):
    """dx, dw, db, and what the roundings of dx and dw go by: r (|g| + mean |g| +
    |h| mean |g h|) and sum |a h|, sum |a|."""
    a = dy.double() + (0.0 if dy_add is None else dy_add.double())
    g = a * (1.0 if w is None else w.double())
    r = r.double()[:, None]
    m1 = g.mean(1, keepdim=True) if center else 0.0
    dx = r * (g - m1 - h * (g * h).mean(1, keepdim=True))
    size = r * (g.abs() + (g.abs().mean(1, keepdim=True) if center else 0.0) + h.abs() * (g * h).abs().mean(1, keepdim=True))
    if dx_add is not None:
        dx = dx + dx_add.double()
        size = size + dx_add.double().abs()
    return dx, (a * h).sum(0), a.sum(0), size, (a * h).abs().sum(0), a.abs().sum(0)


def swiglu(d_act, h_q, h_s):
    """dh, act, and what their roundings go by."""
    h = decode(h_q, h_s)
    F = h.shape[1] // 2
    g, u, a = h[:, :F], h[:, F:], d_act.double()
    sg = torch.sigmoid(g)
    p = g * sg
    dh = torch.cat([a * u * (sg + p * torch.sigmoid(-g)), a * p], 1)
    act = p * u
    # sigmoid: 2^-22 from the exponential, |g| 2^-23 from its argument, 2^-23 from the
    # reciprocal; up to six products and sums of 2^-24 each on top
    rel = 2.0 ** -21 * (1.0 + g.abs() / 4)
    e_dh = torch.cat([rel * (a * u).abs() * (sg + p.abs()), rel * (a * p).abs()], 1)
    return dh, act, e_dh, rel * act.abs()


def padded(v, offsets, pad, ld):
    """Rows of each expert at their padded places, zeros between: [ld, C]."""
    out = v.new_zeros(ld, v.shape[1])
    for e in range(len(offsets) - 1):
        n = offsets[e + 1] - offsets[e]
        out[pad[e]:pad[e] + n] = v[offsets[e]:offsets[e + 1]]
    return out


def pad_offsets(offsets):
    pad = [0]
    for e in range(len(offsets) - 1):
        pad.append(pad[-1] + (offsets[e + 1] - offsets[e] + 127) // 128 * 128)
    return pad
