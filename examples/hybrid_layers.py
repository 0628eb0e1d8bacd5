"""A small stack of linear-attention layers, served: packed prompts, then single tokens.

KDA layers and layers with one decay per head take turns. Between them, every operator of the
library runs as in a served model: ``add_norm`` adds a block's output to the residual stream and
norms it for the next block, the chunked forwards (``fwd``, ``la_fwd``) take the prompts and leave
each sequence's state in the layer's pool, ``step`` and ``la_step`` continue from there token by
token, and ``norm_gate`` norms and gates the heads' outputs. The projections are plain matrix
products with random weights.

    python examples/hybrid_layers.py

decodes a few tokens after the prompts and compares every one with the prompts run again with
those tokens at their end.
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_02_gb300 as kda  # noqa: E402

BF16 = torch.bfloat16


class Layer:
    """One block: projections, a linear attention, the heads' norm and gate, the output projection."""

    def __init__(self, kind, D, H, Hk, K, V, pool_rows, gen):
        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device="cuda") * rows ** -0.5).to(BF16)

        self.kind, self.H, self.Hk, self.K, self.V = kind, H, H if kind == "kda" else Hk, K, V
        self.w_in = weight(D, 2 * self.Hk * K + 2 * H * V)       # q, k, v and the output's gate
        self.w_out = weight(H * V, D)
        self.norm = torch.ones(D, device="cuda")
        self.head_norm = torch.ones(V, device="cuda")
        self.pool = torch.zeros(pool_rows, H, V, K, device="cuda")
        if kind == "kda":
            self.w_g, self.w_beta = weight(D, H * K), weight(D, H)
            self.A_log = torch.zeros(H, device="cuda")
            self.dt_bias = torch.full((H, K), -3.0, device="cuda")
        else:
            self.decay = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)

    def project(self, y):
        x = y @ self.w_in
        q, k, v, z = torch.split(x, [self.Hk * self.K, self.Hk * self.K, self.H * self.V, self.H * self.V], -1)
        return (q.unflatten(-1, (self.Hk, self.K)), k.unflatten(-1, (self.Hk, self.K)),
                v.unflatten(-1, (self.H, self.V)), z.unflatten(-1, (self.H, self.V)))

    def output(self, o, z):
        return kda.norm_gate(o, z, self.head_norm, activation="silu").flatten(-2) @ self.w_out

    def prompt(self, y, cu, rows):
        """y [1,T,D], sequences packed by cu; their last states go to the pool's `rows`."""
        q, k, v, z = self.project(y)
        if self.kind == "kda":   # kda.fwd takes contiguous tensors
            g = (y @ self.w_g).unflatten(-1, (self.H, self.K))
            o, state = kda.fwd(q.contiguous(), k.contiguous(), v.contiguous(), g, y @ self.w_beta, self.A_log,
                               self.dt_bias, -5.0, output_final_state=True, cu_seqlens=cu)
        else:
            o, state = kda.la_fwd(q, k, v, self.decay, output_final_state=True, cu_seqlens=cu)
        self.pool[rows.long()] = state
        return self.output(o, z)

    def token(self, y, rows):
        """y [N,D], one token of each request; the states in the pool's `rows` move on."""
        q, k, v, z = self.project(y)
        if self.kind == "kda":
            g = (y @ self.w_g).unflatten(-1, (self.H, self.K))
            o = kda.step(q, k, v, g, y @ self.w_beta, self.A_log, self.pool, dt_bias=self.dt_bias, state_indices=rows)
        else:
            o = kda.la_step(q, k, v, self.decay, self.pool, state_indices=rows)
        return self.output(o, z)


class Model:
    def __init__(self, D=1024, H=8, Hk=2, K=128, V=128, layers=4, pool_rows=16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.layers = [Layer("kda" if i % 2 == 0 else "la", D, H, Hk, K, V, pool_rows, gen) for i in range(layers)]
        self.last_norm = torch.ones(D, device="cuda")

    def __call__(self, x, run):
        """x: embeddings; run(layer, y): a layer's output. Returns the normed last residual stream."""
        residual, block = x.float(), torch.zeros_like(x)
        for layer in self.layers:
            y, residual = kda.add_norm(block, residual, layer.norm, residual_out=residual)
            block = run(layer, y)
        return kda.add_norm(block, residual, self.last_norm)[0]

    def prompt(self, x, cu, rows):
        return self(x, lambda layer, y: layer.prompt(y, cu, rows))

    def token(self, x, rows):
        return self(x, lambda layer, y: layer.token(y, rows))


def check(lens=(700, 1, 64, 333), tokens=4, D=1024, **kw):
    """Largest rel-L2 difference of a decoded token's output from the longer prompt's."""
    model = Model(D=D, **kw)
    gen = torch.Generator(device="cuda").manual_seed(1)
    seqs = [torch.randn(n + tokens, D, generator=gen, device="cuda").to(BF16) for n in lens]
    rows = torch.tensor([3 * i + 1 for i in range(len(lens))], dtype=torch.int32, device="cuda")

    def pack(extra):
        ends = torch.tensor([0] + [n + extra for n in lens]).cumsum(0).to(torch.int32).cuda()
        return torch.cat([s[:n + extra] for s, n in zip(seqs, lens)])[None], ends

    model.prompt(*pack(0), rows)
    worst = 0.0
    decoded = [model.token(torch.stack([s[n + t] for s, n in zip(seqs, lens)]), rows) for t in range(tokens)]
    for t, y in enumerate(decoded):
        x, ends = pack(t + 1)
        want = model.prompt(x, ends, rows)[0, ends[1:].long() - 1].float()
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    assert kda.device_status() == 0
    return worst


def decode_time(model, N, steps=50):
    """Seconds per token of a batch of N, replayed from a CUDA graph."""
    x = torch.randn(N, model.last_norm.numel(), device="cuda").to(BF16)
    rows = torch.arange(N, dtype=torch.int32, device="cuda")
    model.token(x, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.token(x, rows)
    graph.replay()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    return (time.perf_counter() - t0) / steps


if __name__ == "__main__":
    print(f"decoded tokens against longer prompts: rel-L2 {check():.2e}")
    print(f"4 layers, 16 requests: {1e6 * decode_time(Model(), 16):.0f} us per token")
