"""One decode step of a multi-tenant server's last layer, as an example of how
the serving-step operators run together:

    python -m tenant_lora_serving_amd.decode_step [--rows 256] [--adapters 32] [--context 1000] [--prefix 0]

    s  = x + residual, q8 = norm(s) in e4m3        rms_norm
    qkv = q8 Wqkv^T + adapters                     lora_linear, 8-bit form
    o  = attend(qkv) Wo^T + adapters               lora_linear
    h  = norm(o + s)                               rms_norm
    z  = h Whead^T + adapters                      lora_linear
    log probabilities of the answered tokens       token_logprobs

The attention is `attend`: by default the query columns pass through;
CachedAttention (with --context) keeps every request's keys and values in a
paged cache (kv_append, paged_attention).  Workspaces are made once and used by every step, and a step
allocates nothing that a graph capture cannot hold, so the example captures it
and replays the graph; it prints the time of a step both ways.
"""
from __future__ import annotations

import argparse
import time
from typing import NamedTuple

import torch

from . import step

EPS = 1e-5


class Projection(NamedTuple):
    """A shared weight and every tenant's adapter of it (the `lora` pools' layout)."""
    w: torch.Tensor          # [N, k] bf16 or float8_e4m3fn
    w_scale: object          # [N] float32 with an 8-bit weight, else None
    a_pool: torch.Tensor     # [S, L, R, k] bf16
    b_pool: torch.Tensor     # [S, N, R] bf16
    sizes: tuple             # L slice widths

    def workspace(self, n):
        S, L, R, k = self.a_pool.shape
        return step.linear_workspace(n, k, self.w.shape[0], L, R, self.w.device)


def make_projection(g, k, sizes, slots, rank, quant=False) -> Projection:
    """Random weights and adapters on g's device."""
    def normal(*shape, std):
        return torch.randn(*shape, generator=g, device=g.device) * std

    w, w_scale = normal(sum(sizes), k, std=k ** -0.5), None
    if quant:
        w_scale = w.abs().amax(dim=1) / 448
        w = (w / w_scale[:, None]).to(torch.float8_e4m3fn)
    else:
        w = w.bfloat16()
    return Projection(w, w_scale, normal(slots, len(sizes), rank, k, std=k ** -0.5).bfloat16(),
                      normal(slots, sum(sizes), rank, std=rank ** -0.5).bfloat16(), tuple(sizes))


class CachedAttention:
    """`attend` of a step for up to `rows` requests of up to `context` tokens each, over a paged
    cache: appends every request's new token and attends over all of its tokens and, before
    them, those of the prefix that it shares: request i has prefix i * len(prefixes) // rows.
    `lens`, the tokens that each request has in the cache, lives on the device and grows by one
    a call, in a replayed graph too; a full request's last token is written over."""

    def __init__(self, heads, kv_heads, dim, rows, context, prefixes=(), page=16, quant=False, base=500000.0,
                 device="cuda"):
        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device=device)

        if context < 1 or page < 1 or min(prefixes, default=0) < 0:
            raise ValueError("context and page must be at least 1, prefixes at least 0 tokens long")
        self.heads, self.kv, self.dim, self.page, self.context = heads, kv_heads, dim, page, context
        self.prefixes = tuple(prefixes)
        each, counts = -(-context // page), [-(-p // page) for p in prefixes]
        shape = (2, rows * each + sum(counts), page, kv_heads, dim)
        self.cache = torch.zeros(shape, dtype=torch.bfloat16, device=device)
        self.scales = {}
        if quant:
            self.cache = self.cache.to(torch.float8_e4m3fn)
            self.scales = {name: torch.full((kv_heads,), 1 / 64, device=device) for name in ("k_scale", "v_scale")}
        self.pages = ints(range(rows * each)).view(rows, each)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=device)
        self.before = torch.zeros(rows, dtype=torch.int32, device=device)
        self.prefix = None
        if prefixes:
            firsts = [rows * each + sum(counts[:i]) for i in range(len(counts))]
            tables = [[f + j if j < c else -1 for j in range(max(counts))] for f, c in zip(firsts, counts)]
            starts = [-(-rows * i // len(prefixes)) for i in range(len(prefixes) + 1)]
            self.prefix = step.Prefixes(ints(tables), ints(list(prefixes)), ints(starts))
            self.before = ints([prefixes[i * len(prefixes) // rows] for i in range(rows)])
        self.rotation = step.rotation_table(context + max(prefixes, default=0), dim, base, device)
        self.ws = step.attention_workspace(rows, heads, kv_heads, dim, bool(prefixes), device)

    def parts(self, qkv):
        """q, k and v of a projection's result, [n, heads, dim] each."""
        wide = [h * self.dim for h in (self.heads, self.kv, self.kv)]
        return [p.unflatten(1, (-1, self.dim)) for p in qkv.split(wide, dim=1)]

    def fill_prefix(self, i, qkv):
        """The keys and values of all of prefix i's tokens, from their projection's result."""
        if not 0 <= i < len(self.prefixes):
            raise IndexError(f"there is no prefix {i}")
        if qkv.shape[0] != self.prefixes[i]:
            raise ValueError(f"prefix {i} has {self.prefixes[i]} tokens, got {qkv.shape[0]}")
        _, k, v = self.parts(qkv)
        t = torch.arange(k.shape[0], device=k.device)
        place = self.prefix.pages[i][t // self.page] * self.page + t % self.page
        step.kv_append(k, v, *self.cache, place.int(), positions=t.int(), rotation=self.rotation, **self.scales)

    def __call__(self, qkv):
        n = qkv.shape[0]
        q, k, v = self.parts(qkv)
        at = self.lens[:n].clamp(0, self.context - 1)
        place = self.pages[:n].gather(1, (at // self.page)[:, None].long())[:, 0] * self.page + at % self.page
        q = step.kv_append(k, v, *self.cache, place, q=q, positions=at + self.before[:n], rotation=self.rotation,
                           **self.scales)
        self.lens[:n] = at + 1
        prefix = self.prefix
        if prefix is not None and n < self.lens.shape[0]:   # (the batch is a part of the rows)
            prefix = prefix._replace(starts=prefix.starts.clamp_max(n))
        r = step.paged_attention(q, *self.cache, self.pages[:n], self.lens[:n], prefix=prefix, ws=self.ws, **self.scales)
        return r.out.flatten(1)


class StepResult(NamedTuple):
    norm: step.NormResult
    qkv: torch.Tensor
    attended: torch.Tensor
    o: torch.Tensor
    final: step.NormResult
    logits: torch.Tensor
    scores: step.LogprobResult


class DecodeStep:
    """The step for up to `rows` requests: weights, and workspaces of its own."""

    def __init__(self, hidden, kv, vocab, slots, rank, rows, top=5, seed=0, device="cuda", attend=None):
        g = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.top = hidden, top
        self.attend = attend or (lambda qkv: qkv[:, :hidden])
        self.qkv = make_projection(g, hidden, (hidden, kv, kv), slots, rank, quant=True)
        self.o = make_projection(g, hidden, (hidden,), slots, rank)
        self.head = make_projection(g, hidden, (vocab,), slots, rank)
        self.norms = [(1 + 0.1 * torch.randn(hidden, generator=g, device=device)).bfloat16() for _ in range(2)]
        self.scale = 0.25 + torch.rand(slots, generator=g, device=device)
        self.ws = [p.workspace(rows) for p in (self.qkv, self.o, self.head)]
        self.score_ws = step.logprobs_workspace(rows, vocab, top, device)

    def _project(self, p, ws, x, slot, **kw):
        return step.lora_linear(x, p.w, p.a_pool, p.b_pool, self.scale, p.sizes, slot, ws=ws, **kw)

    def __call__(self, x, residual, slot, tokens) -> StepResult:
        """x, residual [n, hidden] bf16; slot [n] int32, each request's adapter
        (negative: none); tokens [n] int32, the answered tokens."""
        a = step.rms_norm(x, self.norms[0], EPS, residual=residual, quant=True)
        qkv = self._project(self.qkv, self.ws[0], a.y, slot, xq=a.q, x_scale=a.q_scale, w_scale=self.qkv.w_scale)
        attended = self.attend(qkv)
        o = self._project(self.o, self.ws[1], attended, slot)
        f = step.rms_norm(o, self.norms[1], EPS, residual=a.residual)
        logits = self._project(self.head, self.ws[2], f.y, slot)
        scores = step.token_logprobs(logits, tokens, self.top, ws=self.score_ws)
        return StepResult(a, qkv, attended, o, f, logits, scores)


def main():
    ap = argparse.ArgumentParser(description="times one decode step of the serving-step operators")
    ap.add_argument("--rows", type=int, default=256)
    ap.add_argument("--adapters", type=int, default=32)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--context", type=int, default=0, help="tokens of a request in the cache at most; 0: no attention")
    ap.add_argument("--prefix", type=int, default=0, help="tokens of a prefix that all requests share")
    args = ap.parse_args()
    if args.context < 0 or args.prefix < 0 or (args.prefix > 0 and args.context == 0):
        ap.error("--context and --prefix are lengths, and --prefix needs a --context")
    n = args.rows
    g = torch.Generator(device="cuda").manual_seed(1)
    attend = None
    if args.context:
        attend = CachedAttention(32, 8, 128, n, args.context, (args.prefix,) if args.prefix else ())
        attend.cache.normal_(generator=g)
        attend.lens.copy_(torch.randint(0, args.context, (n,), generator=g, device="cuda"))
    run = DecodeStep(4096, 1024, 128256, args.adapters, args.rank, n, attend=attend)
    x, residual = (torch.randn(n, 4096, generator=g, device="cuda").bfloat16() for _ in range(2))
    slot = torch.randint(0, args.adapters, (n,), generator=g, device="cuda").to(torch.int32)
    tokens = torch.randint(0, 128256, (n,), generator=g, device="cuda").to(torch.int32)

    def timed(f, reps=50):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / reps * 1e6

    eager = timed(lambda: run(x, residual, slot, tokens))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = run(x, residual, slot, tokens)
    replay = timed(graph.replay)
    print(f"{n} rows, {args.adapters} adapters of rank {args.rank}: {eager:.1f} us a step, {replay:.1f} us as a graph")
    for i in range(min(n, 3)):
        print(f"row {i}: log p {r.scores.logprob[i].item():.3f}, rank {r.scores.rank[i].item()}, most likely "
              f"{r.scores.top_ids[i].tolist()}")


if __name__ == "__main__":
    main()
