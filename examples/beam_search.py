"""Beam search with a small Mamba-2 stack, end to end on the library's operators.

A prompt goes through ``ssd_conv_fwd`` and ``ssd_fwd`` layer by layer, which
leaves every layer's convolution ring and state; each further token goes through
``ssd_w4_matvec`` (the projections, 4-bit weights), ``ssd_step``,
``ssd_beam_select`` and ``ssd_beam_reorder`` (the rings and states follow the
beams).  Weights are random: the program shows how the calls fit together.

    python examples/beam_search.py [--batch 2] [--beams 4] [--prompt 37] [--tokens 16]
"""
import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import mamba_ssd_forward_chunked_gb300 as ssd  # noqa: E402

HEADDIM, CHUNK = 64, 64


class W4Linear:
    """A projection with 4-bit weights."""

    def __init__(self, rows, cols, g, group=64, device="cuda"):
        weight = torch.randn(rows, cols, generator=g) / cols ** 0.5
        self.packed, self.scales = (t.to(device) for t in ssd.w4_quantize(weight, group))
        self.group = group

    def __call__(self, x, add=None):
        return ssd.ssd_w4_matvec(x, self.packed, self.scales, self.group, add=add)


class Layer:
    """x + out(gate * ssd(conv(in(norm(x))))): one Mamba-2 layer."""

    def __init__(self, width, g, dstate=64, ngroups=1, taps=4, device="cuda"):
        self.nheads, self.dstate, self.ngroups, self.taps = 2 * width // HEADDIM, dstate, ngroups, taps
        self.inner, self.gn = self.nheads * HEADDIM, ngroups * dstate
        self.channels = self.inner + 2 * self.gn
        put = lambda t: t.to(device)  # noqa: E731
        self.proj_in = W4Linear(self.inner + self.channels + self.nheads, width, g, device=device)
        self.proj_out = W4Linear(width, self.inner, g, device=device)
        self.weight, self.bias = put(torch.rand(self.channels, taps, generator=g) - 0.5), put(torch.zeros(self.channels))
        self.A = put(-torch.exp(torch.rand(self.nheads, generator=g) * 2.77))
        self.D = put(torch.ones(self.nheads))
        dt = torch.exp(torch.rand(self.nheads, generator=g) * 4.6 - 6.9)
        self.dt_bias = put(dt + torch.log(-torch.expm1(-dt)))

    def cache(self, rows, dtype):
        """(ring, state) for that many sequences."""
        return (torch.zeros(rows, self.taps, self.channels, dtype=dtype, device=self.A.device),
                torch.zeros(rows, self.nheads, HEADDIM, self.dstate, device=self.A.device))

    def _split(self, proj):
        """z, the convolution's input and dt, side by side in the projection."""
        return proj.split([self.inner, self.channels, self.nheads], dim=-1)

    def prompt(self, x, ring):
        """x [B, L, width] -> (x after the layer, final state); the ring is filled."""
        B, L, width = x.shape
        z, u, dt = self._split(self.proj_in(_norm(x).view(B * L, width)).view(B, L, -1))
        xs, Bm, Cm = ssd.ssd_conv_fwd(u, self.weight, self.bias, split=(self.inner, self.gn, self.gn), ring=ring)
        y, state = ssd.ssd_fwd(xs.view(B, L, self.nheads, HEADDIM),
                               torch.nn.functional.softplus(dt.float() + self.dt_bias), self.A,
                               Bm.view(B, L, self.ngroups, self.dstate), Cm.view(B, L, self.ngroups, self.dstate),
                               self.D, CHUNK)
        y = (y.view(B, L, self.inner).float() * torch.nn.functional.silu(z.float())).to(x.dtype)
        return self.proj_out(y.view(B * L, self.inner), add=x.view(B * L, width)).view(B, L, width), state

    def step(self, x, ring, state, positions):
        """x [B, width], one token each -> x after the layer; ring and state take the token."""
        z, u, dt = self._split(self.proj_in(_norm(x)))
        y = ssd.ssd_step(u, dt, self.A, self.D, self.weight, self.bias, state, ring, positions, ngroups=self.ngroups,
                         z=z, dt_bias=self.dt_bias, dt_softplus=True)
        return self.proj_out(y.view(-1, self.inner), add=x)


def _norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)


class Model:
    def __init__(self, vocab=1000, width=128, layers=2, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.dtype = dtype
        self.embed = torch.randn(vocab, width, generator=g).to(device, dtype)
        self.layers = [Layer(width, g, device=device) for _ in range(layers)]
        self.head = W4Linear(vocab, width, g, device=device)

    def prompt(self, tokens):
        """tokens [B, L] -> (logits of every position [B, L, V], one (ring, state) a layer)."""
        x, caches = self.embed[tokens], []
        for layer in self.layers:
            ring, _ = layer.cache(tokens.shape[0], self.dtype)
            x, state = layer.prompt(x, ring)
            caches.append((ring, state))
        B, L, width = x.shape
        return self.head(_norm(x).view(B * L, width)).view(B, L, -1), caches

    def step(self, tokens, caches, positions):
        """tokens [N] -> logits [N, V]; the caches take the token."""
        x = self.embed[tokens]
        for layer, (ring, state) in zip(self.layers, caches):
            x = layer.step(x, ring, state, positions)
        return self.head(_norm(x))


def beam_search(model, prompt, beams, steps, eos):
    """prompt [B, L] -> (tokens [B, beams, steps], scores [B, beams]), best first."""
    B, L = prompt.shape
    logits, caches = model.prompt(prompt)
    scores, _, tokens = ssd.ssd_beam_select(logits[:, -1:], torch.zeros(B, 1, device=prompt.device), beams)
    # every request's one cache row becomes `beams` rows
    flat = [t for pair in caches for t in pair]
    wide = [t.new_empty(B * beams, *t.shape[1:]) for t in flat]
    ssd.ssd_beam_reorder(flat, torch.zeros(B, beams, dtype=torch.int32, device=prompt.device), out=wide)
    caches = list(zip(wide[0::2], wide[1::2]))
    history = tokens[:, :, None]
    for t in range(steps - 1):
        positions = torch.full((B * beams,), L + t, dtype=torch.int32, device=prompt.device)
        logits = model.step(tokens.reshape(-1), caches, positions)
        scores, parents, tokens = ssd.ssd_beam_select(logits.view(B, beams, -1), scores, beams,
                                                      finished=(history == eos).any(-1), eos=eos)
        ssd.ssd_beam_reorder([t for pair in caches for t in pair], parents)
        history = torch.cat([history.gather(1, parents.long()[..., None].expand_as(history)), tokens[:, :, None]], -1)
    return history, scores


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=37)
    ap.add_argument("--tokens", type=int, default=16)
    args = ap.parse_args()
    model = Model()
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(0, 1000, (args.batch, args.prompt), generator=g).cuda()
    beam_search(model, prompt, args.beams, args.tokens, eos=0)
    torch.cuda.synchronize()
    began = time.perf_counter()
    tokens, scores = beam_search(model, prompt, args.beams, args.tokens, eos=0)
    torch.cuda.synchronize()
    took = time.perf_counter() - began
    for b in range(args.batch):
        for w in range(args.beams):
            print(f"request {b} beam {w}: {float(scores[b, w]):9.4f}  {tokens[b, w].tolist()}")
    print(f"{args.batch} requests x {args.beams} beams, {args.tokens} tokens in {took * 1e3:.2f} ms")


if __name__ == "__main__":
    main()
