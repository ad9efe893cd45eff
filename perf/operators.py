"""Timing cases of the operators that serve a Mamba layer around ``ssd_fwd``.

Five operators: the short causal convolution (``ssd_conv_fwd``), the selective
scan with a decay per channel and state (``ssd_selective_scan``, prompts and
single tokens), the single-token Mamba-2 step (``ssd_step``), products of a few
tokens with 4-bit weights (``ssd_w4_matvec``), and beam search's selection with
the reordering of the states it decides (``ssd_beam_select``,
``ssd_beam_reorder``).

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs on the
GPU, ``run()`` one pass: the plain torch form where ``own`` is false, the
framework's entry points where it is true.  ``work()`` counts a pass's
compulsory bytes and operations and ``exact()`` computes the outputs in 64
bits, from the definitions.
"""
import math

import torch

own = False

HEADDIM = 64


def _ssd():
    import mamba_ssd_forward_chunked_gb300 as ssd
    return ssd


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the Mamba-2 2.7B layer's prompt: x, B and C out of the in-projection's output
        dict(name="conv-prompt-2.7b", op="conv", batch=4, seqlen=4096, nheads=80, dstate=128, ngroups=1, width=4,
             resume=False, ragged=False, dtype="bf16"),
        # the 370M layer, a prompt of odd length taken up again from its ring, sequences of different lengths
        dict(name="conv-resumed-ragged", op="conv", batch=3, seqlen=1021, nheads=32, dstate=128, ngroups=1, width=4,
             resume=True, ragged=True, dtype="f32"),
        # a batch of prompts with as many channels as the 2.7B layer
        dict(name="scan-prompt", op="scan", batch=2, seqlen=2048, channels=5120, dstate=16, ngroups=1, gate=True,
             ragged=False, dtype="bf16"),
        # one long sequence with the 370M layer's channels: too few channels to fill the GPU by themselves
        dict(name="scan-long", op="scan", batch=1, seqlen=16384, channels=2048, dstate=16, ngroups=1, gate=False,
             ragged=False, dtype="f32"),
        # decoding: one token of 64 sequences
        dict(name="scan-token", op="scan", batch=64, seqlen=1, channels=5120, dstate=16, ngroups=1, gate=True,
             ragged=False, dtype="bf16"),
        # decoding one sequence through the 2.7B layer: latency
        dict(name="step-one", op="step", batch=1, nheads=80, dstate=128, ngroups=1, width=4, dtype="bf16"),
        # decoding a full batch: the states' bandwidth
        dict(name="step-batch", op="step", batch=256, nheads=80, dstate=128, ngroups=1, width=4, dtype="bf16"),
        # the 2.7B layer's in-projection for one token
        dict(name="w4-in-one", op="w4", tokens=1, k=2560, n=10576, group=128, add=False, dtype="bf16"),
        # its out-projection onto the residual stream for eight sequences
        dict(name="w4-out-eight", op="w4", tokens=8, k=5120, n=2560, group=64, add=True, dtype="bf16"),
        # odd sizes, 32-bit activations, a last group that ends early
        dict(name="w4-odd", op="w4", tokens=3, k=1001, n=1777, group=32, add=False, dtype="f32"),
        # one request, four beams, with the 370M layer's state of one layer
        dict(name="beam-one", op="beam", batch=1, beams=4, vocab=32768, nheads=32, dstate=128, finished=False,
             dtype="f32"),
        # many requests and a large vocabulary, some beams finished
        dict(name="beam-batch", op="beam", batch=32, beams=8, vocab=131072, nheads=8, dstate=128, finished=True,
             dtype="bf16"),
    ]


def _spread(rng, low, high):
    """An odd size between low and high, evenly spread over its logarithm."""
    return max(1, int(round(math.exp(rng.uniform(math.log(low), math.log(high))))) | 1)


def draw(rng):
    op = rng.choice(["conv", "scan", "step", "w4", "beam"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "conv":
        seqlen = _spread(rng, 1, 16384)
        nheads = rng.choice([8, 16, 32, 64, 80])
        most = max(1, 44_000_000 // (seqlen * nheads * HEADDIM))
        return dict(op=op, batch=min(most, rng.choice([1, 2, 3, 5, 8, 64])), seqlen=seqlen, nheads=nheads,
                    dstate=rng.choice([64, 128]), ngroups=rng.choice([1, 2]), width=rng.choice([2, 3, 4]),
                    resume=rng.random() < 0.5, ragged=rng.random() < 0.5, dtype=dtype)
    if op == "scan":
        seqlen = 1 if rng.random() < 0.25 else _spread(rng, 2, 16384)
        ngroups = rng.choice([1, 1, 2])
        channels = ngroups * 8 * _spread(rng, 32, 640)
        dstate = rng.choice([8, 13, 16, 16, 16, 32, 64])
        most = max(1, 330_000_000 // (seqlen * channels * dstate))
        return dict(op=op, batch=min(most, rng.choice([1, 2, 3, 8, 64])), seqlen=min(seqlen, 330_000_000 // (channels * dstate)),
                    channels=channels, dstate=dstate, ngroups=ngroups, gate=rng.random() < 0.5,
                    ragged=rng.random() < 0.5, dtype=dtype)
    if op == "step":
        return dict(op=op, batch=_spread(rng, 1, 200), nheads=rng.choice([8, 16, 32, 64, 80]),
                    dstate=rng.choice([64, 128]), ngroups=rng.choice([1, 2]), width=rng.choice([2, 3, 4]), dtype=dtype)
    if op == "w4":
        k = _spread(rng, 64, 8192) if rng.random() < 0.5 else 64 * _spread(rng, 4, 100)
        return dict(op=op, tokens=rng.randint(1, 16), k=k, n=_spread(rng, 64, 16384), group=rng.choice([32, 64, 128]),
                    add=rng.random() < 0.5, dtype=dtype)
    vocab = _spread(rng, 1000, 131072)
    return dict(op=op, batch=min(rng.choice([1, 2, 4, 9, 32]), max(1, 16_000_000 // (8 * vocab))), beams=rng.choice([1, 2, 3, 4, 5, 8]),
                vocab=vocab, nheads=rng.choice([4, 8, 32]), dstate=rng.choice([64, 128]),
                finished=rng.random() < 0.5, dtype=dtype)


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


def _prepare_conv(case, r):
    B, L, W = case["batch"], case["seqlen"], case["width"]
    inner, gn = case["nheads"] * HEADDIM, case["ngroups"] * case["dstate"]
    C = inner + 2 * gn
    proj = r.normal(B, L, 2 * inner + 2 * gn + case["nheads"], dtype=_dtype(case))  # z | x B C | dt
    s = dict(u=proj[:, :, inner:inner + C], weight=r.uniform(-0.5, 0.5, C, W), bias=r.uniform(-0.5, 0.5, C),
             split=(inner, gn, gn), ring=r.normal(B, W, C, dtype=_dtype(case)), positions=None, lengths=None)
    s["new_ring"] = torch.empty_like(s["ring"])
    s["positions"] = r.ints(0, 5000, B) if case["resume"] else torch.zeros(B, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        s["lengths"] = r.ints(0, L + 1, B)
        s["lengths"][0] = L
    return s


def _prepare_scan(case, r):
    B, L, D, N, G = case["batch"], case["seqlen"], case["channels"], case["dstate"], case["ngroups"]
    dt = _dtype(case)
    bc = r.normal(B, L, 2 * G * N, dtype=dt)  # B and C side by side, as their projection leaves them
    s = dict(u=r.normal(B, L, D, dtype=dt), delta=r.normal(B, L, D, dtype=dt).mul_(0.5), delta_bias=r.dt_bias(D),
             A=-torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * r.normal(D, N)),
             Bm=bc[:, :, :G * N].unflatten(2, (G, N)), Cm=bc[:, :, G * N:].unflatten(2, (G, N)), D=r.normal(D),
             z=r.normal(B, L, D, dtype=dt) if case["gate"] else None, init=r.normal(B, D, N), lengths=None)
    if case["ragged"]:
        s["lengths"] = r.ints(0, L + 1, B)
        s["lengths"][0] = L
    return s


def _prepare_step(case, r):
    B, H, N, G, W = case["batch"], case["nheads"], case["dstate"], case["ngroups"], case["width"]
    inner, gn = H * HEADDIM, G * N
    C = inner + 2 * gn
    proj = r.normal(B, 2 * inner + 2 * gn + H, dtype=_dtype(case))  # z | x B C | dt
    s = dict(u=proj[:, inner:inner + C], z=proj[:, :inner], dt=proj[:, inner + C:], dt_bias=r.dt_bias(H),
             A=-torch.exp(r.uniform(0.0, math.log(16.0), H)), D=r.normal(H), weight=r.uniform(-0.5, 0.5, C, W),
             bias=r.uniform(-0.5, 0.5, C), ring=r.normal(B, W, C, dtype=_dtype(case)),
             state=r.normal(B, H, HEADDIM, N).mul_(0.3), positions=r.ints(0, 5000, B), ngroups=G,
             slots=torch.randperm(B, generator=r.g, device="cuda").to(torch.int32))
    s["new_state"] = torch.empty_like(s["state"])
    return s


def _pack(codes):
    """4-bit codes [n, k] in the order the product reads them: tiles of 16 rows
    and 64 columns, 32 lanes of four words each (include/ssd.h, ssd_w4_matvec)."""
    n, k = codes.shape
    nt, kt = -(-n // 16), -(-k // 64)
    full = torch.full((nt * 16, kt * 64), 8, dtype=torch.int32, device=codes.device)
    full[:n, :k] = codes
    # row = tile, half (bit 2 j of the shift), r; column = tile, half, c, word, pair (bit of the shift), place
    v = full.view(nt, 2, 8, kt, 2, 4, 2, 2, 2).permute(0, 3, 2, 5, 4, 6, 7, 1, 8)
    shift = torch.tensor([[[0, 16], [4, 20]], [[8, 24], [12, 28]]], dtype=torch.int64, device=codes.device)
    words = (v.to(torch.int64) << shift).sum(dim=(-3, -2, -1))
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    return words.to(torch.int32).reshape(nt, kt, 32, 4)


def _prepare_w4(case, r):
    M, K, N, g = case["tokens"], case["k"], case["n"], case["group"]
    codes = r.ints(0, 16, N, K, dtype=torch.uint8)
    return dict(x=r.normal(M, K, dtype=_dtype(case)), codes=codes, packed=_pack(codes), group=g,
                scales=r.uniform(0.5, 1.5, N, -(-K // g)).mul_(1.0 / math.sqrt(20.0 * K)),
                add=r.normal(M, N, dtype=_dtype(case)) if case["add"] else None)


def _prepare_beam(case, r):
    B, W, V, H, N = case["batch"], case["beams"], case["vocab"], case["nheads"], case["dstate"]
    C = H * HEADDIM + 2 * N
    s = dict(logits=r.normal(B, W, V, dtype=_dtype(case)).mul_(3.0), scores=r.uniform(-30.0, -20.0, B, W).sort(1, True)[0],
             eos=2, finished=None, state=r.normal(B * W, H, HEADDIM, N), ring=r.normal(B * W, 4, C, dtype=_dtype(case)))
    s["logits"][:, :, 7] = -math.inf  # a token that is never allowed
    if case["finished"]:
        s["finished"] = r.uniform(0.0, 1.0, B, W) < 0.2
    s["new"] = [torch.empty_like(s["state"]), torch.empty_like(s["ring"])]
    return s


def prepare(case, seed):
    r = _Rand(seed)
    s = {"conv": _prepare_conv, "scan": _prepare_scan, "step": _prepare_step, "w4": _prepare_w4,
         "beam": _prepare_beam}[case["op"]](case, r)
    s["op"] = case["op"]
    return s


# ------------------------------------------------------------------ plain forms

def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20.0, v, torch.log1p(torch.exp(torch.clamp(v, max=20.0))))


def _plain_window(u, weight, bias, ring, positions):
    """Convolution with silu of u [B, L, C] in 32 bits after the ring's tokens."""
    L, W = u.shape[1], weight.shape[1]
    back = positions.long()[:, None] + torch.arange(1 - W, 0, device=u.device)  # the W-1 tokens before
    rows = torch.arange(u.shape[0], device=u.device)[:, None]
    before = torch.where((back >= 0)[..., None], ring.float()[rows, back % W], 0.0)
    taps = torch.cat([before, u], 1).unfold(1, W, 1)  # [B, L, C, W]
    return _silu((taps * weight).sum(-1) + bias)


def _plain_ring(u, ring, positions, lengths):
    """The ring after the tokens of u: every slot's newest token."""
    W, L = ring.shape[1], u.shape[1]
    last = (positions.long() + lengths - 1)[:, None]
    token = last - (last - torch.arange(W, device=u.device)) % W  # newest token of each slot
    i = token - positions.long()[:, None]
    rows = torch.arange(u.shape[0], device=u.device)[:, None]
    return torch.where((i >= 0)[..., None], u[rows, i.clamp(0, L - 1)], ring)


def _plain_conv(s):
    u = s["u"]
    B, L, _ = u.shape
    y = _plain_window(u.float(), s["weight"], s["bias"], s["ring"], s["positions"])
    lengths = torch.full((B,), L, device=u.device) if s["lengths"] is None else s["lengths"].long()
    y = torch.where((torch.arange(L, device=u.device) < lengths[:, None])[..., None], y, 0.0).to(u.dtype)
    parts = [p.contiguous() for p in y.split(s["split"], dim=2)]
    return parts + [_plain_ring(u, s["ring"], s["positions"], lengths)]


def _plain_scan(s):
    """The recurrence over all tokens at once, by doubling: after a round of
    width w every entry holds the last 2 w tokens' joint decay and input."""
    u, z, L, G = s["u"].float(), s["z"], s["u"].shape[1], s["Bm"].shape[2]
    per = u.shape[2] // G
    d = _softplus(s["delta"].float() + s["delta_bias"])
    if s["lengths"] is not None:
        live = (torch.arange(L, device=u.device) < s["lengths"][:, None])[..., None]
        d = torch.where(live, d, 0.0)
    Bm = s["Bm"].float().repeat_interleave(per, 2)
    Cm = s["Cm"].float().repeat_interleave(per, 2)
    a = torch.exp(d[..., None] * s["A"])
    h = (d * u)[..., None] * Bm
    h[:, 0] += a[:, 0] * s["init"]
    w = 1
    while w < L:
        h = torch.cat([h[:, :w], h[:, w:] + a[:, w:] * h[:, :-w]], 1)
        a = torch.cat([a[:, :w], a[:, w:] * a[:, :-w]], 1)
        w *= 2
    y = (h * Cm).sum(-1) + s["D"] * u
    if z is not None:
        y = y * _silu(z.float())
    if s["lengths"] is not None:
        y = torch.where(live, y, 0.0)
    return [y.to(s["u"].dtype), h[:, -1].contiguous()]


def _plain_step(s):
    B, H, P, N = s["state"].shape
    G, W, slots = s["ngroups"], s["ring"].shape[1], s["slots"].long()
    u = s["u"][:, None]
    xbc = _plain_window(u.float(), s["weight"], s["bias"], s["ring"][slots], s["positions"])[:, 0]
    x = xbc[:, :H * P].view(B, H, P)
    Bm = xbc[:, H * P:H * P + G * N].view(B, G, N).repeat_interleave(H // G, 1)
    Cm = xbc[:, H * P + G * N:].view(B, G, N).repeat_interleave(H // G, 1)
    d = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(d * s["A"])[..., None, None] * s["state"][slots] + (d[..., None] * x)[..., None] * Bm[:, :, None]
    y = (h * Cm[:, :, None]).sum(-1) + s["D"][:, None] * x
    y = y * _silu(s["z"].float()).view(B, H, P)
    new_state, ring = torch.empty_like(s["state"]), s["ring"].clone()
    new_state[slots] = h
    ring[slots, s["positions"].long() % W] = s["u"]
    return [y.to(s["u"].dtype), new_state, ring]


def _plain_w4(s):
    K = s["x"].shape[1]
    w = (s["codes"].float() - 8.0) * s["scales"].repeat_interleave(s["group"], 1)[:, :K]
    y = torch.matmul(s["x"].float(), w.t())
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(s["x"].dtype)


def _candidates(x, scores, finished, eos):
    """Every candidate's score, [batch, beams, vocab], in x's type."""
    top = x.amax(-1, keepdim=True)
    log_sum = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    c = scores[..., None] + (x - log_sum)
    c = torch.where(torch.isnan(c), -math.inf, c)
    if finished is not None:
        stay = torch.full_like(c, -math.inf)
        stay[..., eos] = scores
        c = torch.where(finished[..., None], stay, c)
    return c


def _plain_beam(s):
    B, W, V = s["logits"].shape
    c = _candidates(s["logits"].float(), s["scores"], s["finished"], s["eos"])
    best, at = c.view(B, W * V).sort(dim=1, descending=True, stable=True)
    best, at = best[:, :W].contiguous(), at[:, :W]
    parents, tokens = (at // V).to(torch.int32), (at % V).to(torch.int32)
    rows = (torch.arange(B, device=at.device)[:, None] * W + parents).view(-1)
    return [best, parents, tokens, s["state"][rows], s["ring"][rows]]


# ------------------------------------------------------------------ the framework's operators

def _own_conv(s):
    parts = _ssd().ssd_conv_fwd(s["u"], s["weight"], s["bias"], activation="silu", split=s["split"], ring=s["ring"],
                                positions=s["positions"], lengths=s["lengths"], new_ring=s["new_ring"])
    return list(parts) + [s["new_ring"]]


def _own_scan(s):
    return list(_ssd().ssd_selective_scan(s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], z=s["z"],
                                          delta_bias=s["delta_bias"], delta_softplus=True, init_state=s["init"],
                                          lengths=s["lengths"]))


def _own_step(s):
    y = _ssd().ssd_step(s["u"], s["dt"], s["A"], s["D"], s["weight"], s["bias"], s["state"], s["ring"], s["positions"],
                        ngroups=s["ngroups"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, slots=s["slots"],
                        new_state=s["new_state"])
    return [y, s["new_state"], s["ring"]]


def _own_w4(s):
    return _ssd().ssd_w4_matvec(s["x"], s["packed"], s["scales"], s["group"], add=s["add"])


def _own_beam(s):
    ssd = _ssd()
    best, parents, tokens = ssd.ssd_beam_select(s["logits"], s["scores"], s["logits"].shape[1], finished=s["finished"],
                                                eos=s["eos"])
    ssd.ssd_beam_reorder([s["state"], s["ring"]], parents, out=s["new"])
    return [best, parents, tokens] + s["new"]


_PLAIN = {"conv": _plain_conv, "scan": _plain_scan, "step": _plain_step, "w4": _plain_w4, "beam": _plain_beam}
_OWN = {"conv": _own_conv, "scan": _own_scan, "step": _own_step, "w4": _own_w4, "beam": _own_beam}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "conv":
        C = case["nheads"] * HEADDIM + 2 * case["ngroups"] * case["dstate"]
        n = case["batch"] * case["seqlen"] * C
        W = case["width"]
        rings = case["batch"] * W * C * es * (2 if case["resume"] else 1)
        return {"bytes": 2 * n * es + rings + C * (W + 1) * 4, "flops": n * (2 * W + 5)}
    if op == "scan":
        B, L, D, N, G = (case[k] for k in ("batch", "seqlen", "channels", "dstate", "ngroups"))
        n = B * L * D
        return {"bytes": n * es * (4 if case["gate"] else 3) + 2 * B * L * G * N * es + 2 * B * D * N * 4 + D * N * 4 + 8 * D,
                "flops": n * (7 * N + 10)}
    if op == "step":
        B, H, N, G = (case[k] for k in ("batch", "nheads", "dstate", "ngroups"))
        C = H * HEADDIM + 2 * G * N
        state = B * H * HEADDIM * N
        return {"bytes": 8 * state + B * es * ((case["width"] + 1) * C + 2 * H * HEADDIM + H) + C * (case["width"] + 1) * 4,
                "flops": 5 * state + B * C * (2 * case["width"] + 5)}
    if op == "w4":
        M, K, N = case["tokens"], case["k"], case["n"]
        return {"bytes": N * K // 2 + N * -(-K // case["group"]) * 4 + M * K * es + M * N * es * (2 if case["add"] else 1),
                "flops": 2 * M * N * K}
    rows = case["batch"] * case["beams"]
    row = case["nheads"] * HEADDIM * case["dstate"] * 4 + 4 * (case["nheads"] * HEADDIM + 2 * case["dstate"]) * es
    return {"bytes": rows * case["vocab"] * es + 2 * rows * row + 16 * rows, "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_taps(u, weight, bias, ring, positions):
    """The convolution with silu, one tap after the other, u [B, L, C] in 64 bits."""
    B, L, C = u.shape
    W = weight.shape[1]
    ext = torch.zeros(B, L + W - 1, C, dtype=torch.float64, device=u.device)
    ext[:, W - 1:] = u
    for b, p in enumerate(positions.tolist()):
        for j in range(1, min(W - 1, p) + 1):
            ext[b, W - 1 - j] = ring[b, (p - j) % W].double()
    acc = bias.double().expand(B, L, C).clone()
    for j in range(W):
        acc += weight[:, j].double() * ext[:, j:j + L]
    return acc * torch.sigmoid(acc)


def _exact_conv(s):
    u = s["u"].double()
    y = _exact_taps(u, s["weight"], s["bias"], s["ring"], s["positions"])
    ring = s["ring"].double().clone()
    W = ring.shape[1]
    lengths = [u.shape[1]] * u.shape[0] if s["lengths"] is None else s["lengths"].tolist()
    for b, (p, n) in enumerate(zip(s["positions"].tolist(), lengths)):
        y[b, n:] = 0.0
        for t in range(max(0, n - W), n):
            ring[b, (p + t) % W] = u[b, t]
    a, g, _ = s["split"]
    return [y[..., :a].contiguous(), y[..., a:a + g].contiguous(), y[..., a + g:].contiguous(), ring]


def _exact_scan(s):
    B, L, D = s["u"].shape
    G = s["Bm"].shape[2]
    A, h = s["A"].double(), s["init"].double().clone()
    y = torch.zeros(B, L, D, dtype=torch.float64, device=h.device)
    lengths = torch.full((B,), L, device=h.device) if s["lengths"] is None else s["lengths"].long()
    for t in range(L):
        d = torch.nn.functional.softplus(s["delta"][:, t].double() + s["delta_bias"].double(), threshold=60.0)
        ut = s["u"][:, t].double()
        Bt = s["Bm"][:, t].double().repeat_interleave(D // G, 1)
        Ct = s["Cm"][:, t].double().repeat_interleave(D // G, 1)
        new = torch.exp(d[..., None] * A) * h + (d * ut)[..., None] * Bt
        yt = torch.einsum("bdn,bdn->bd", new, Ct) + s["D"].double() * ut
        if s["z"] is not None:
            zt = s["z"][:, t].double()
            yt = yt * zt * torch.sigmoid(zt)
        live = (t < lengths)[:, None]
        h = torch.where(live[..., None], new, h)
        y[:, t] = torch.where(live, yt, 0.0)
    return [y, h]


def _exact_step(s):
    B, H, P, N = s["state"].shape
    G, slots = s["ngroups"], s["slots"].long()
    xbc = _exact_taps(s["u"].double()[:, None], s["weight"], s["bias"], s["ring"][slots], s["positions"])[:, 0]
    x, Bm, Cm = xbc.split([H * P, G * N, G * N], dim=1)
    x, Bm, Cm = x.view(B, G, H // G, P), Bm.view(B, G, N), Cm.view(B, G, N)
    d = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=60.0)
    h = s["state"][slots].double() * torch.exp(d * s["A"].double())[..., None, None]
    h = h + torch.einsum("bgkp,bgn->bgkpn", d.view(B, G, H // G, 1) * x, Bm).reshape(B, H, P, N)
    y = torch.einsum("bgkpn,bgn->bgkp", h.view(B, G, H // G, P, N), Cm).reshape(B, H, P)
    y = y + s["D"].double()[:, None] * x.reshape(B, H, P)
    z = s["z"].double().view(B, H, P)
    new_state = torch.empty_like(h)
    new_state[slots] = h
    ring = s["ring"].double().clone()
    ring[slots, s["positions"].long() % ring.shape[1]] = s["u"].double()
    return [y * z * torch.sigmoid(z), new_state, ring]


def _exact_w4(s):
    K, g = s["x"].shape[1], s["group"]
    y = torch.zeros(s["x"].shape[0], s["codes"].shape[0], dtype=torch.float64, device="cuda")
    for i, k in enumerate(range(0, K, g)):
        part = s["x"][:, k:k + g].double() @ (s["codes"][:, k:k + g].double() - 8.0).t()
        y += part * s["scales"][:, i].double()
    return y if s["add"] is None else y + s["add"].double()


def _exact_beam(s):
    B, W, V = s["logits"].shape
    best = []
    for b in range(B):
        x = s["logits"][b].double()
        c = s["scores"][b].double()[:, None] + torch.log_softmax(x, -1)
        if s["finished"] is not None:
            for w in torch.nonzero(s["finished"][b]).flatten().tolist():
                c[w] = -math.inf
                c[w, s["eos"]] = s["scores"][b, w].double()
        best.append(c.flatten().topk(W)[0])
    return [torch.stack(best), None, None, None, None]


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "step": _exact_step, "w4": _exact_w4,
            "beam": _exact_beam}[case["op"]](s)
