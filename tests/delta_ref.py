"""64-bit references of the gated delta rule and of the verification of drafted
tokens, from the formulas in include/ssd.h: torch double on the CPU, one token
after the other.

Bound of the delta rule.  A token takes a row s of a head's state to
    s' = a s (I - beta k k^T) + beta x k^T,
so an error e of the row becomes at most m a |e| with m = max(1, |1 - beta |k|^2|),
the norm of I - beta k k^T, and the token's own roundings add at most
EPS (a |s| + beta |k| (|x| + 2 a |s| |k|)): each product and sum is off by a few
units of 2^-24, the gates and the norms of k by a few more, EPS (layer_ref) being
16.  In chunks of C tokens the values that are written come out of a triangular
system whose inverse has entries of at most m^C beta |k|^2: an error of one
token's value reaches the C - 1 after it, each by that much, so `spread` is 1 + C
there.  An output is off by |scale| |q| times the state's error and EPS of the
state's norm; in chunks, where it is the entering state's part plus
sum_j (P T)_tj r_j, also by P T's rounding to 11 bits (bf16) or 22, pt |(P T)_tj| |r_j|.
(P T)_tj is scale q_t.z_j, z_j being k_j carried through the tokens after j."""
import torch

from layer_ref import EPS, HALF_BF16, d64, softplus


def delta(x, dt, A, Bm, Cm, beta, scale=None, dt_bias=None, dt_softplus=False, beta_sigmoid=False, norm_eps=None,
          init_state=None, slots=None, positions=None, lengths=None, final_state=None, spread=1.0, eps=EPS, pt=2.0 ** -12):
    """(y, its bound, final state, its bound); rows of final_state that no
    sequence has are those of ``final_state`` (0)."""
    x, dt, A, Bm, Cm, beta = (d64(v) for v in (x, dt, A, Bm, Cm, beta))
    B, L, H, P = x.shape
    G, N = Bm.shape[2:]
    if dt_bias is not None:
        dt = dt + d64(dt_bias)
    if dt_softplus:
        dt = softplus(dt)
    if beta_sigmoid:
        beta = torch.sigmoid(beta)
    if norm_eps is not None:
        Bm = Bm * torch.where((Bm.square().sum(-1, keepdim=True) + norm_eps) > 0, (Bm.square().sum(-1, keepdim=True) + norm_eps).rsqrt(), 0.0)
        Cm = Cm * torch.where((Cm.square().sum(-1, keepdim=True) + norm_eps) > 0, (Cm.square().sum(-1, keepdim=True) + norm_eps).rsqrt(), 0.0)
    scale = N ** -0.5 if scale is None else scale
    S = B if init_state is None and final_state is None else (init_state if init_state is not None else final_state).shape[0]
    out = torch.zeros(S, H, P, N, dtype=torch.float64) if final_state is None else d64(final_state).clone()
    err = torch.zeros_like(out)
    y, ybound = torch.zeros(B, L, H, P, dtype=torch.float64), torch.zeros(B, L, H, P, dtype=torch.float64)
    for b in range(B):
        row = b if slots is None else int(slots[b])
        if not 0 <= row < S:
            continue
        h = torch.zeros(H, P, N, dtype=torch.float64)
        if init_state is not None and (positions is None or int(positions[b]) > 0):
            h = d64(init_state)[row].clone()
        e = torch.zeros(H, P, dtype=torch.float64)
        carried, rests, entering = [], [], h
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for t in range(n):
            k, q = Bm[b, t].repeat_interleave(H // G, 0), Cm[b, t].repeat_interleave(H // G, 0)
            a, w, kn = torch.exp(dt[b, t] * A), beta[b, t], k.norm(dim=-1)
            # the argument of the exponential has a rounding of its own
            size = a[:, None] * h.norm(dim=-1) * (1 + (dt[b, t] * A).abs()[:, None])
            own = eps * (size + (w.abs() * kn)[:, None] * (x[b, t].abs() + 2 * size * kn[:, None]))
            m = torch.maximum((1 - w * kn * kn).abs(), torch.ones_like(w))
            e = (m * a)[:, None] * e + spread * own
            if spread > 1:
                if t % 64 == 0:
                    carried, rests, entering = [], [], h
                entering = entering * a[:, None, None]
                rests.append(w[:, None] * (x[b, t] - (entering * k[:, None]).sum(-1)))
                carried = [a[:, None] * (z - (w * (z * k).sum(-1))[:, None] * k) for z in carried] + [k]
            h = h * a[:, None, None]
            h = h + (w[:, None] * (x[b, t] - (h * k[:, None]).sum(-1)))[..., None] * k[:, None]
            y[b, t] = scale * (h * q[:, None]).sum(-1)
            for z, r in zip(carried, rests):
                ybound[b, t] += pt * abs(scale) * (q * z).sum(-1).abs()[:, None] * r.abs()
            ybound[b, t] += abs(scale) * q.norm(dim=-1)[:, None] * (e + eps * h.norm(dim=-1))
        out[row], err[row] = h, e[..., None].expand(H, P, N)
    return y, ybound, out, err + 2.0 ** -23 * out.abs() + 1e-30


def verify(logits, draft, uniforms, draft_logits=None, scale=None, lengths=None):
    """(tokens, accepted, log-probabilities): a loop over each sequence's drafts."""
    logits, u = d64(logits), d64(uniforms)
    B, T1, V = logits.shape
    T = T1 - 1
    tokens, accepted = torch.full((B, T1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    logprobs = torch.zeros(B, T1, dtype=torch.float64)

    def shares(row, s):
        row = torch.where(torch.isnan(row), -float("inf"), row)
        top = row.max()
        if top == -float("inf"):
            return torch.zeros(V, dtype=torch.float64)
        w = torch.exp(torch.where(row == top, 0.0, (row - top) * s))
        return w / w.sum()

    for b in range(B):
        s = 1.0 if scale is None else float(scale[b])
        if not 0.0 < s < float("inf"):
            continue
        count = T if lengths is None else min(max(int(lengths[b]), 0), T)
        n, q = 0, None
        while True:
            p = shares(logits[b, n], s)
            if n == count:
                q = torch.zeros(V, dtype=torch.float64)
                break
            d = int(draft[b, n])
            known = 0 <= d < V
            if draft_logits is None:
                q = torch.zeros(V, dtype=torch.float64)
                if known:
                    q[d] = 1.0
            else:
                q = shares(d64(draft_logits)[b, n], s)
            if not known or not u[b, n] * q[d] < p[d]:
                break
            tokens[b, n], logprobs[b, n] = d, p[d].log()
            n += 1
        accepted[b] = n
        rest = (p - q).clamp(min=0.0)
        if not bool(rest.sum() > 0):
            rest = p
        if bool(rest.sum() > 0):
            c = rest.cumsum(0)
            v = min(int((c <= u[b, T] * c[-1]).sum()), V - 1)
            tokens[b, n], logprobs[b, n] = v, p[v].log()
    return tokens, accepted, logprobs


__all__ = ["EPS", "HALF_BF16", "d64", "delta", "verify"]
