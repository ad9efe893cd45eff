"""Timing cases of the gated delta rule and of the verification of drafted tokens.

Two operators: the recurrence with a gated delta rule (``ssd_delta_fwd``: whole
prompts, a few drafted tokens and single tokens), and the verification of drafted
tokens against the target's probabilities with given random numbers
(``ssd_draft_verify``), whose counts are the lengths that the recurrence commits.

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs on the
GPU, ``run()`` one pass: the plain torch form where ``own`` is false, the
framework's entry points where it is true.  ``work()`` counts a pass's
compulsory bytes and operations and ``exact()`` computes the outputs in 64
bits, from the definitions.
"""
import math

import torch

own = False

NORM_EPS = 1e-6


def _ssd():
    import mamba_ssd_forward_chunked_gb300 as ssd
    return ssd


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a batch of prompts; two value heads share a key head
        dict(name="delta-prompt", op="delta", batch=4, seqlen=4096, nheads=32, ngroups=16, headdim=128, dstate=128,
             cached=False, ragged=False, dtype="bf16"),
        # one long sequence with few heads: nothing but the chain of its tokens
        dict(name="delta-long", op="delta", batch=1, seqlen=16384, nheads=16, ngroups=16, headdim=128, dstate=128,
             cached=False, ragged=False, dtype="bf16"),
        # prompts of odd lengths taken up again from cached states, small heads
        dict(name="delta-resumed-ragged", op="delta", batch=3, seqlen=1021, nheads=16, ngroups=8, headdim=64, dstate=64,
             cached=True, ragged=True, dtype="bf16"),
        # 32-bit activations
        dict(name="delta-f32", op="delta", batch=2, seqlen=501, nheads=8, ngroups=4, headdim=128, dstate=128,
             cached=True, ragged=True, dtype="f32"),
        # the last token and four drafted ones of 32 sequences, as many of them as were accepted
        dict(name="delta-drafts", op="delta", batch=32, seqlen=5, nheads=32, ngroups=16, headdim=128, dstate=128,
             cached=True, ragged=True, dtype="bf16"),
        # decoding one sequence: latency
        dict(name="delta-token-one", op="delta", batch=1, seqlen=1, nheads=32, ngroups=16, headdim=128, dstate=128,
             cached=True, ragged=False, dtype="bf16"),
        # decoding a full batch: the states' bandwidth
        dict(name="delta-token-batch", op="delta", batch=256, seqlen=1, nheads=32, ngroups=16, headdim=128, dstate=128,
             cached=True, ragged=False, dtype="bf16"),
        # one request, four drafted tokens
        dict(name="verify-one", op="verify", batch=1, drafts=4, vocab=32768, probs=True, scaled=False, ragged=False,
             dtype="f32"),
        # many requests and a large vocabulary, a temperature for each
        dict(name="verify-batch", op="verify", batch=32, drafts=7, vocab=131072, probs=True, scaled=True, ragged=False,
             dtype="bf16"),
        # drafts looked up instead of drawn (no draft model), an odd vocabulary, different numbers of drafts
        dict(name="verify-lookup", op="verify", batch=64, drafts=3, vocab=50001, probs=False, scaled=False, ragged=True,
             dtype="bf16"),
    ]


def _spread(rng, low, high):
    """An odd size between low and high, evenly spread over its logarithm."""
    return max(1, int(round(math.exp(rng.uniform(math.log(low), math.log(high))))) | 1)


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.6:
        seqlen = 1 if rng.random() < 0.2 else _spread(rng, 2, 16384)
        nheads = rng.choice([4, 6, 8, 16, 32])
        headdim, dstate = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
        most = max(1, (8_000_000_000 if dtype == "bf16" else 1_000_000_000) // (seqlen * nheads * headdim * dstate))
        return dict(op="delta", batch=min(most, rng.choice([1, 2, 3, 5, 8, 61, 200])), seqlen=seqlen, nheads=nheads,
                    ngroups=nheads // rng.choice([1, 2]), headdim=headdim, dstate=dstate, cached=rng.random() < 0.6,
                    ragged=rng.random() < 0.5, dtype=dtype)
    vocab, drafts = _spread(rng, 1000, 131072), rng.randint(1, 8)
    most = max(1, 30_000_000 // (vocab * (drafts + 1)))
    return dict(op="verify", batch=min(most, rng.choice([1, 2, 4, 9, 32, 64])), drafts=drafts, vocab=vocab,
                probs=rng.random() < 0.7, scaled=rng.random() < 0.5, ragged=rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------------ inputs

class _Rand:
    """Seeded values on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=self.g, device="cuda", dtype=dtype)

    def uniform(self, low, high, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda") * (high - low) + low

    def ints(self, low, high, *shape, dtype=torch.int32):
        return torch.randint(low, high, shape, generator=self.g, device="cuda", dtype=dtype)

    def dt_bias(self, n):
        """Biases whose softplus is a step between 0.001 and 0.1, log-uniform."""
        dt = torch.exp(self.uniform(math.log(1e-3), math.log(0.1), n))
        return dt + torch.log(-torch.expm1(-dt))


def _prepare_delta(case, r):
    B, L, H, G, P, N = (case[k] for k in ("batch", "seqlen", "nheads", "ngroups", "headdim", "dstate"))
    dt = _dtype(case)
    gates = r.normal(B, L, 2 * H, dtype=dt)  # dt | beta, as their projection leaves them
    s = dict(x=r.normal(B, L, H, P, dtype=dt), Bm=r.normal(B, L, G, N, dtype=dt), Cm=r.normal(B, L, G, N, dtype=dt),
             dt=gates[:, :, :H], beta=gates[:, :, H:], dt_bias=r.dt_bias(H),
             A=-torch.exp(r.uniform(0.0, math.log(16.0), H)), init=None, slots=None, positions=None, lengths=None)
    S = B
    if case["cached"]:  # rows of a cache, one of them belonging to a sequence that begins
        S = B + 3
        s["init"] = r.normal(S, H, P, N).mul_(0.3)
        s["slots"] = torch.randperm(S, generator=r.g, device="cuda")[:B].to(torch.int32)
        s["positions"] = r.ints(1, 5000, B)
        if B > 1:
            s["positions"][B // 2] = 0
    if case["ragged"]:
        s["lengths"] = r.ints(0, L + 1, B)
        s["lengths"][0] = L
    s["final"] = torch.zeros(S, H, P, N, device="cuda")
    return s


def _prepare_verify(case, r):
    B, T, V = case["batch"], case["drafts"], case["vocab"]
    target = r.normal(B, T + 1, V).mul_(3.0)
    target[:, :, 7] = -math.inf  # a token that is never allowed
    if case["probs"]:  # drawn from a draft model that is near the target
        near = target[:, :T] + r.normal(B, T, V).mul_(0.6)
        draft = (near - torch.log(-torch.log(r.uniform(1e-7, 1.0, B, T, V)))).argmax(-1)
        near = near.to(_dtype(case))
    else:  # looked up: often what the target expects too
        draft, near = r.ints(8, V, B, T, dtype=torch.int64), None
        target[:, :T].scatter_add_(2, draft[..., None], r.uniform(5.0, 25.0, B, T, 1))
    s = dict(logits=target.to(_dtype(case)), draft=draft.to(torch.int32), draft_logits=near,
             uniforms=torch.rand(B, T + 1, generator=r.g, device="cuda"), scale=None, lengths=None)
    if case["scaled"]:
        s["scale"] = 1.0 / r.uniform(0.6, 1.4, B)
    if case["ragged"]:
        s["lengths"] = r.ints(0, T + 1, B)
    return s


def prepare(case, seed):
    r = _Rand(seed)
    s = {"delta": _prepare_delta, "verify": _prepare_verify}[case["op"]](case, r)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------ plain forms

def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _unit(v):
    return v / torch.sqrt((v * v).sum(-1, keepdim=True) + NORM_EPS)


def _inverse(A):
    """(I + A)^-1 for strictly lower triangular A [..., C, C], C a power of two:
    diagonal blocks of twice the size a round, [[X, 0], [-Y A21 X, Y]]."""
    C = A.shape[-1]
    T = torch.eye(C, device=A.device).expand_as(A).contiguous()
    place = torch.arange(C, device=A.device)
    size = 1
    while size < C:
        below = (place[:, None] // size == place // size + 1) & (place // size % 2 == 0)
        T = T - torch.matmul(T, torch.matmul(torch.where(below, A, 0.0), T))
        size *= 2
    return T


def _chunks(v, C):
    """[B, L, H, ...] as [B, H, chunks, C, ...], zeros after the last token."""
    B, L, H = v.shape[:3]
    n = -(-L // C)
    full = v.new_zeros(B, n * C, *v.shape[2:])
    full[:, :L] = v
    return full.view(B, n, C, *v.shape[2:]).movedim(3, 1)


def _plain_delta(s):
    """Chunk by chunk: within a chunk the rule is a triangular system."""
    x, init = s["x"], s["init"]
    B, L, H, P = x.shape
    G, N = s["Bm"].shape[2:]
    g = _softplus(s["dt"].float() + s["dt_bias"]) * s["A"]
    beta = 1.0 / (1.0 + torch.exp(-s["beta"].float()))
    live = torch.ones(B, L, dtype=torch.bool, device=x.device)
    if s["lengths"] is not None:
        live = torch.arange(L, device=x.device) < s["lengths"][:, None]
        g, beta = torch.where(live[..., None], g, 0.0), torch.where(live[..., None], beta, 0.0)
    C = min(64, 1 << (L - 1).bit_length())
    v = _chunks(x.float(), C)
    k = _chunks(_unit(s["Bm"].float()), C).repeat_interleave(H // G, 1)
    q = _chunks(_unit(s["Cm"].float()), C).repeat_interleave(H // G, 1) * N ** -0.5
    beta = _chunks(beta, C)[..., None]
    total = _chunks(g.double(), C).cumsum(-1)  # differences of long sums
    at = torch.arange(C, device=x.device)
    decay = torch.where(at[:, None] >= at, total[..., None] - total[..., None, :], -math.inf).exp().float()
    since = total.exp().float()[..., None]
    until = (total[..., -1:] - total).exp().float()[..., None]
    T = _inverse(torch.where(at[:, None] > at, beta * decay * torch.matmul(k, k.transpose(-1, -2)), 0.0))
    u, w = torch.matmul(T, beta * v), torch.matmul(T, beta * since * k)
    inside = decay * torch.matmul(q, k.transpose(-1, -2))
    S = torch.zeros(B, H, N, P, device=x.device)
    rows = torch.arange(B, device=x.device)
    if init is not None:
        rows = s["slots"].long()
        S = torch.where((s["positions"] > 0)[:, None, None, None], init[rows], 0.0).transpose(-1, -2)
    y = torch.empty_like(v)
    for c in range(v.shape[2]):
        new = u[:, :, c] - torch.matmul(w[:, :, c], S)
        y[:, :, c] = since[:, :, c] * torch.matmul(q[:, :, c], S) + torch.matmul(inside[:, :, c], new)
        S = since[:, :, c, -1:] * S + torch.matmul((until[:, :, c] * k[:, :, c]).transpose(-1, -2), new)
    y = y.flatten(2, 3)[:, :, :L].transpose(1, 2)
    final = torch.zeros_like(s["final"])
    final[rows] = S.transpose(-1, -2)
    return [torch.where(live[..., None, None], y, 0.0).to(x.dtype), final]


def _probabilities(logits, scale):
    """softmax over the vocabulary in 64 bits."""
    v = logits.double() * scale
    e = torch.exp(v - v.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _plain_verify(s):
    """In 64 bits: which token a random number hits depends on sums over the vocabulary."""
    logits, draft, u = s["logits"], s["draft"].long(), s["uniforms"].double()
    B, T = draft.shape
    scale = torch.ones(B, 1, 1, device=u.device, dtype=torch.float64)
    if s["scale"] is not None:
        scale = s["scale"].double()[:, None, None]
    p = _probabilities(logits, scale)
    q = torch.zeros_like(p)
    if s["draft_logits"] is not None:
        q[:, :T] = _probabilities(s["draft_logits"], scale)
    else:
        q[:, :T].scatter_(2, draft[..., None], 1.0)
    at = draft[..., None]
    taken = (u[:, :T, None] * q[:, :T].gather(2, at) < p[:, :T].gather(2, at))[..., 0]
    count = torch.full((B, 1), T, device=u.device) if s["lengths"] is None else s["lengths"].long()[:, None]
    place = torch.arange(T + 1, device=u.device)
    taken = taken & (place[:T] < count)
    accepted = taken.long().cumprod(1).sum(1, keepdim=True)
    rows = torch.arange(B, device=u.device)
    last, drafted = p[rows, accepted[:, 0]], q[rows, accepted[:, 0]]
    drafted = torch.where(accepted < count, drafted, 0.0)
    rest = torch.clamp(last - drafted, min=0.0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0.0, rest, last)
    total = rest.cumsum(-1)
    token = (total <= u[:, T:] * total[:, -1:]).sum(-1, keepdim=True)
    full = torch.cat([draft, draft.new_zeros(B, 1)], 1)
    tokens = torch.where(place < accepted, full, torch.where(place == accepted, token, -1))
    chosen = torch.log(p.gather(2, tokens.clamp(min=0)[..., None]))[..., 0]
    return [tokens.to(torch.int32), accepted[:, 0].to(torch.int32), torch.where(tokens >= 0, chosen, 0.0).float()]


# ------------------------------------------------------------------ the framework's operators

def _own_delta(s):
    y, final = _ssd().ssd_delta_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["beta"], dt_bias=s["dt_bias"],
                                    dt_softplus=True, beta_sigmoid=True, norm_eps=NORM_EPS, init_state=s["init"],
                                    slots=s["slots"], positions=s["positions"], lengths=s["lengths"],
                                    final_state=s["final"])
    return [y, final]


def _own_verify(s):
    return list(_ssd().ssd_draft_verify(s["logits"], s["draft"], s["uniforms"], draft_logits=s["draft_logits"],
                                        scale=s["scale"], lengths=s["lengths"]))


_PLAIN = {"delta": _plain_delta, "verify": _plain_verify}
_OWN = {"delta": _own_delta, "verify": _own_verify}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "delta":
        B, L, H, G, P, N = (case[k] for k in ("batch", "seqlen", "nheads", "ngroups", "headdim", "dstate"))
        token = 2 * H * P + 2 * G * N + 2 * H  # x, y; Bm, Cm; dt, beta
        return {"bytes": B * L * token * es + B * H * P * N * 4 * (2 if case["cached"] else 1) + 8 * H,
                "flops": B * L * H * P * N * 7}  # decay, S k, the update, S q
    rows = case["batch"] * (case["drafts"] + 1 + (case["drafts"] if case["probs"] else 0))
    return {"bytes": rows * case["vocab"] * es + case["batch"] * (case["drafts"] + 1) * 16,
            "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_delta(s):
    """The recurrence token by token."""
    B, L, H, P = s["x"].shape
    G, N = s["Bm"].shape[2:]
    h = torch.zeros(B, H, P, N, dtype=torch.float64, device="cuda")
    out = torch.zeros(s["final"].shape, dtype=torch.float64, device="cuda")
    row = list(range(B)) if s["slots"] is None else s["slots"].tolist()
    if s["init"] is not None:
        for b, at in enumerate(s["positions"].tolist()):
            if at > 0:
                h[b] = s["init"][row[b]].double()
    d = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=60.0)
    gate, beta = torch.exp(d * s["A"].double()), torch.sigmoid(s["beta"].double())
    lengths = torch.full((B,), L, device="cuda") if s["lengths"] is None else s["lengths"].long()
    y = torch.zeros(B, L, H, P, dtype=torch.float64, device="cuda")
    for t in range(int(lengths.max())):
        k, q = s["Bm"][:, t].double(), s["Cm"][:, t].double()
        k = (k / (k.square().sum(-1, keepdim=True) + NORM_EPS).sqrt()).repeat_interleave(H // G, 1)
        q = (q / (q.square().sum(-1, keepdim=True) + NORM_EPS).sqrt()).repeat_interleave(H // G, 1) / math.sqrt(N)
        new = h * gate[:, t, :, None, None]
        miss = s["x"][:, t].double() - torch.einsum("bhpn,bhn->bhp", new, k)
        new = new + (beta[:, t, :, None] * miss)[..., None] * k[:, :, None]
        live = t < lengths
        h = torch.where(live[:, None, None, None], new, h)
        y[:, t] = torch.where(live[:, None, None], torch.einsum("bhpn,bhn->bhp", new, q), 0.0)
    for b in range(B):
        out[row[b]] = h[b]
    return [y, out]


def _exact_verify(s):
    """The log-probabilities of the tokens that a loop over each sequence's drafts emits."""
    B, T = s["draft"].shape
    V = s["logits"].shape[2]
    found = torch.zeros(B, T + 1, dtype=torch.float64, device="cuda")
    for b in range(B):
        scale = 1.0 if s["scale"] is None else float(s["scale"][b])
        count = T if s["lengths"] is None else int(s["lengths"][b])
        logp = torch.log_softmax(s["logits"][b].double() * scale, -1)
        n, u = 0, s["uniforms"][b].double()
        while n < count:
            d = int(s["draft"][b, n])
            if s["draft_logits"] is None:
                q = torch.nn.functional.one_hot(torch.tensor(d, device="cuda"), V).double()
            else:
                q = torch.softmax(s["draft_logits"][b, n].double() * scale, -1)
            if not bool(u[n] * q[d] < logp[n, d].exp()):
                break
            found[b, n] = logp[n, d]
            n += 1
        rest = logp[n].exp() if n == count else (logp[n].exp() - q).clamp(min=0.0)
        if float(rest.sum()) == 0.0:
            rest = logp[n].exp()
        total = rest.cumsum(0)
        found[b, n] = logp[n, int(torch.searchsorted(total, u[T] * total[-1], right=True))]
    return [None, None, found]


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "verify": _exact_verify}[case["op"]](s)
