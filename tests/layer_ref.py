"""64-bit references of the layer operators, with the bounds that 32-bit
arithmetic keeps.  Everything here is torch double on the CPU, one token after
the other, from the formulas in include/ssd.h.

EPS is what one step of a sum or one elementary function may lose: 2^-20, eight
units in the last place of a 32-bit number, covers the two or three roundings of
a multiply-add, an exponential (2 units, plus its argument's rounding, which the
bounds count separately) and the softplus or silu around it."""
import torch

EPS = 2.0 ** -20
HALF_BF16 = 2.0 ** -8  # rounding to bfloat16: half a unit is 2^-9, doubled for a sum near a tie


def d64(t):
    return None if t is None else t.detach().cpu().double()


def store(ref, bound, dtype):
    """Adds the rounding to the output's type to a bound."""
    return bound + (HALF_BF16 * ref.abs() if dtype == torch.bfloat16 else 2.0 ** -23 * ref.abs()) + 1e-30


def check(name, got, ref, bound):
    got = d64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), (name, "over the bound by", float(over.max()), "at", int(over.argmax()),
                               "ratio", float(((got - ref).abs() / bound).max()))


def silu(v):
    return v * torch.sigmoid(v)


def silu_err(v, e):
    """Error of silu(v) where v is off by e: its slope is below 1.1."""
    return 1.1 * e + EPS * (1 + v.abs()) * v.abs()


def softplus(v):
    return torch.where(v > 0, v + torch.log1p(torch.exp(-v.abs())), torch.log1p(torch.exp(v)))


def conv(u, weight, bias, ring=None, positions=None, lengths=None, slots=None, act=True):
    """(y, bound, ring after)."""
    u, weight, bias = d64(u), d64(weight), d64(bias)
    B, L, C = u.shape
    W = weight.shape[1]
    old = d64(ring)
    ring = None if ring is None else d64(ring).clone()
    y, bound = torch.zeros(B, L, C, dtype=torch.float64), torch.zeros(B, L, C, dtype=torch.float64)
    for b in range(B):
        pos = 0 if positions is None else max(0, int(positions[b]))
        n = L if lengths is None else min(L, max(0, int(lengths[b])))
        row = b if slots is None else int(slots[b])
        if ring is not None and not 0 <= row < ring.shape[0]:
            continue

        def tap(t):
            if t >= 0:
                return u[b, t]
            if old is None or pos + t < 0:
                return torch.zeros(C, dtype=torch.float64)
            return old[row, (pos + t) % W]
        for t in range(n):
            acc = torch.zeros(C, dtype=torch.float64) if bias is None else bias.clone()
            mag = acc.abs()
            for j in range(W):
                v = weight[:, j] * tap(t - W + 1 + j)
                acc, mag = acc + v, mag + v.abs()
            y[b, t] = silu(acc) if act else acc
            bound[b, t] = silu_err(acc, EPS * mag) if act else EPS * mag
        if ring is not None:
            for t in range(max(0, n - W), n):
                ring[row, (pos + t) % W] = u[b, t]
    return y, bound, ring


def scan(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, use_softplus=False, init=None, lengths=None):
    """(y, bound, state, bound).  The state's error follows the recurrence: each
    step adds EPS (1 + |d A|) of what the absolute terms sum to."""
    u, delta, A, Bm, Cm, D, z, delta_bias, init = (d64(t) for t in (u, delta, A, Bm, Cm, D, z, delta_bias, init))
    B, L, C = u.shape
    N, G = A.shape[1], Bm.shape[2]
    h = torch.zeros(B, C, N, dtype=torch.float64) if init is None else init.clone()
    mag, err = h.abs(), torch.zeros_like(h)
    y, bound = torch.zeros(B, L, C, dtype=torch.float64), torch.zeros(B, L, C, dtype=torch.float64)
    for t in range(L):
        d = delta[:, t] if delta_bias is None else delta[:, t] + delta_bias
        # a softplus argument v is off by its rounding, and the value relatively by (1 + |v|) EPS
        slack = 1 + d.abs() if use_softplus else torch.ones_like(d)
        if use_softplus:
            d = softplus(d)
        Bt, Ct = Bm[:, t].repeat_interleave(C // G, 1), Cm[:, t].repeat_interleave(C // G, 1)
        a = torch.exp(d[..., None] * A)
        x = (d * u[:, t])[..., None] * Bt
        nh, nm = a * h + x, a * mag + x.abs()
        ne = a * err + EPS * (slack[..., None] + slack[..., None] * (d[..., None] * A).abs()) * nm
        yt = (nh * Ct).sum(-1)
        ey = (ne * Ct.abs()).sum(-1) + EPS * (nh * Ct).abs().sum(-1)
        if D is not None:
            yt, ey = yt + D * u[:, t], ey + EPS * (D * u[:, t]).abs()
        if z is not None:
            s = silu(z[:, t])
            ey = ey * s.abs() + yt.abs() * silu_err(z[:, t], 0.0)
            yt = yt * s
        for b in range(B):
            if lengths is None or t < int(lengths[b]):
                h[b], mag[b], err[b], y[b, t], bound[b, t] = nh[b], nm[b], ne[b], yt[b], ey[b]
    return y, bound, h, err


def step(u, dt, A, D, weight, bias, state, ring, positions, ngroups, z=None, dt_bias=None, use_softplus=False,
         slots=None):
    """(y, bound, state, bound, ring)."""
    B = u.shape[0]
    S, H, P, N = state.shape
    G = ngroups
    rows = list(range(B)) if slots is None else [int(s) for s in slots]
    xbc, exbc, ring = conv(u[:, None], weight, bias, ring, positions, None, slots)
    xbc, exbc = xbc[:, 0], exbc[:, 0]
    dt, A, D, z, dt_bias, old = (d64(t) for t in (dt, A, D, z, dt_bias, state))
    new, bnew = old.clone(), torch.zeros_like(old)
    y, by = torch.zeros(B, H, P, dtype=torch.float64), torch.zeros(B, H, P, dtype=torch.float64)
    for b, row in enumerate(rows):
        if not 0 <= row < S:
            continue
        split = [H * P, G * N, G * N]
        (x, Bv, Cv), (ex, eB, eC) = xbc[b].split(split), exbc[b].split(split)
        x, ex = x.view(H, P, 1), ex.view(H, P, 1)
        Bv, eB, Cv, eC = (t.view(G, 1, N).repeat_interleave(H // G, 0) for t in (Bv, eB, Cv, eC))
        d = dt[b] if dt_bias is None else dt[b] + dt_bias
        slack = 1 + d.abs() if use_softplus else torch.ones_like(d)
        d = (softplus(d) if use_softplus else d).view(H, 1, 1)
        slack = slack.view(H, 1, 1)
        dA = d * A.view(H, 1, 1)
        h = torch.exp(dA) * old[row] + d * x * Bv
        mag = torch.exp(dA) * old[row].abs() + (d * x * Bv).abs()
        eh = EPS * slack * (1 + dA.abs()) * mag + d * (ex * Bv.abs() + x.abs() * eB + ex * eB)
        yt = (h * Cv).sum(-1) + D.view(H, 1) * x[..., 0]
        ey = (eh * Cv.abs() + h.abs() * eC + eh * eC + EPS * (h * Cv).abs()).sum(-1)
        ey = ey + D.abs().view(H, 1) * (ex[..., 0] + EPS * x[..., 0].abs())
        if z is not None:
            zz = z[b].view(H, P)
            ey = ey * silu(zz).abs() + yt.abs() * silu_err(zz, 0.0)
            yt = yt * silu(zz)
        y[b], by[b], new[row], bnew[row] = yt, ey, h, eh
    return y, by, new, bnew, ring


def w4(x, codes, scales, group, add=None):
    """(y, bound).  A product passes at most k/16 + 32 additions."""
    x, codes, scales, add = d64(x), d64(codes), d64(scales), d64(add)
    k = x.shape[1]
    w = (codes - 8) * scales.repeat_interleave(group, 1)[:, :k]
    y, bound = x @ w.t(), (k / 16 + 32) * 2.0 ** -23 * (x.abs() @ w.abs().t())
    if add is not None:
        y, bound = y + add, bound + 2.0 ** -23 * (y.abs() + add.abs())
    return y, bound


def beam(logits, scores, k, finished=None, eos=-1):
    """(scores, parents, tokens) with ties by rising flat index."""
    x, s = d64(logits), d64(scores)
    B, W, V = x.shape
    top = x.amax(-1, keepdim=True)
    c = s[..., None] + (x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))))
    if finished is not None:
        only = torch.full_like(c, -float("inf"))
        only[..., eos] = s
        c = torch.where(finished.cpu()[..., None], only, c)
    c = torch.where(torch.isnan(c), -float("inf"), c).reshape(B, W * V)
    best, at = c.sort(dim=1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    return best, at // V, at % V
