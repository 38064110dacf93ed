"""The paged cache's operators run together: a decode step with attention over its own cache, token
by token, against the definition in 64 bits, as a graph, and against whole prompts."""
import math
import subprocess
import sys

import pytest
import torch

from tenant_lora_serving_amd import step
from tenant_lora_serving_amd.decode_step import CachedAttention, DecodeStep
from test_gpu_attend import gen, near

pytestmark = pytest.mark.gpu
HEADS, KV, DIM = 8, 2, 64


def turn(x, positions, rotation):
    row = rotation.double()[positions][:, None, :]
    cos, sin = row.chunk(2, dim=-1)
    a, b = x.double().chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


class Plain:
    """Every request's turned keys and its values in 64 bits, in lists, and what the cache holds of them."""

    def __init__(self, attend, rows):
        self.a, self.k, self.v = attend, [[] for _ in range(rows)], [[] for _ in range(rows)]

    def put(self, i, k, v, position):
        self.k[i].append(turn(k[None], torch.tensor([position], device="cuda"), self.a.rotation)[0])
        self.v[i].append(v.double())

    def held(self, i):
        """The request's keys and values in the cache, each within a rounding (2^-8 in bf16; 2^-4, or half of the
        smallest step, in e4m3) and the turning's fp32 of what was put there."""
        a, tables = self.a, []
        if a.prefix is not None:
            p = i * a.prefix.lens.shape[0] // len(self.k)
            tables.append((a.prefix.pages[p], a.prefix.lens[p].item()))
        tables.append((a.pages[i], a.lens[i].item()))
        got = []
        for cache, put, name in zip(a.cache, (self.k[i], self.v[i]), ("k_scale", "v_scale")):
            x = torch.cat([cache.double()[t[:-(-n // a.page)].long()].flatten(0, 1)[:n] for t, n in tables])
            scale = a.scales[name].double()[:, None] if a.scales else 1.0
            put = torch.stack(put)
            tol = put.abs() * (2.0 ** -4 if a.scales else 2.0 ** -8) + 2.0 ** -20 + (2.0 ** -10 * scale if a.scales else 0)
            assert ((x * scale - put).abs() <= tol).all()
            got.append((x * scale).repeat_interleave(HEADS // KV, dim=1))
        return got

    def attend(self, i, q, position):
        """(o, bound): the result's rounding and p's to bf16; and a turned q that fp32 rounds to the other neighbour, a
        whole step of 2^-7, which a score and so p are off by in proportion to the magnitudes of its terms."""
        k, v = self.held(i)
        q = turn(q[None], torch.tensor([position], device="cuda"), self.a.rotation)[0].bfloat16().double()
        s = (q[None] * k).sum(dim=2) / math.sqrt(DIM)
        p = torch.softmax(s, dim=0)
        off = torch.expm1(2 * (q[None] * k).abs().sum(dim=2).amax(dim=0) / math.sqrt(DIM) * 2.0 ** -7)
        o = (p[:, :, None] * v).sum(dim=0)
        mean = (p[:, :, None] * v.abs()).sum(dim=0)
        return o, 2.0 ** -8 * o.abs() + mean * (2.0 ** -8 + off[:, None])


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("prefixes", [(), (40, 7)])
def test_token_by_token(quant, prefixes):
    rows, steps = 5, 40
    g = gen(1)
    a = CachedAttention(HEADS, KV, DIM, rows, steps, prefixes, quant=quant)
    plain = Plain(a, rows)
    for p, length in enumerate(prefixes):
        qkv = torch.randn(length, (HEADS + 2 * KV) * DIM, generator=g, device="cuda").bfloat16()
        a.fill_prefix(p, qkv)
        _, k, v = a.parts(qkv)
        for i in range(rows):
            if i * len(prefixes) // rows == p:
                for t in range(length):
                    plain.put(i, k[t], v[t], t)
    for t in range(steps):
        qkv = torch.randn(rows, (HEADS + 2 * KV) * DIM, generator=g, device="cuda").bfloat16()
        got = a(qkv).view(rows, HEADS, DIM)
        q, k, v = a.parts(qkv)
        for i in range(rows):
            before = a.before[i].item()
            plain.put(i, k[i], v[i], before + t)
            if t % 8 == 0 or t == steps - 1:
                want, tol = plain.attend(i, q[i], before + t)
                near(got[i], want, tol, f"token {t} of request {i}")
    assert a.lens.tolist() == [steps] * rows


@pytest.mark.parametrize("quant", [False, True])
def test_prompt_and_tokens_give_the_same(quant):
    """A prompt's rows at once, and its tokens one by one, over the same cache."""
    n = 150
    g = gen(2)
    a = CachedAttention(HEADS, KV, DIM, 1, n, (), quant=quant)
    qkv = torch.randn(n, (HEADS + 2 * KV) * DIM, generator=g, device="cuda").bfloat16()
    one = torch.cat([a(qkv[t:t + 1]) for t in range(n)]).view(n, HEADS, DIM)
    q, k, v = a.parts(qkv)
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    b = CachedAttention(HEADS, KV, DIM, 1, n, (), quant=quant)
    turned = step.kv_append(k, v, *b.cache, t, q=q, positions=t, rotation=b.rotation, **b.scales)
    assert torch.equal(a.cache.view(torch.uint8), b.cache.view(torch.uint8))
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for max_rows in (1, n):
        r = step.paged_attention(turned, *b.cache, b.pages, torch.full((1,), n, dtype=torch.int32, device="cuda"),
                                 starts=starts, max_rows=max_rows, **b.scales)
        # each within its own rounding and p's (sum p |v| <= max |v|) of the same value
        values = v.double().abs().amax() * (1 + 2.0 ** -4)
        bound = 2 * 2.0 ** -8 * (one.double().abs() + 1.02 * values)
        near(r.out, one.double(), bound, "prompt")


@pytest.mark.parametrize("prefixes", [(), (33,)])
def test_step_as_a_graph(prefixes):
    hidden, kv, vocab, slots, n = HEADS * DIM, KV * DIM, 2000, 4, 9
    g = gen(3)

    def make():
        a = CachedAttention(HEADS, KV, DIM, n, 50, prefixes)
        if prefixes:
            a.fill_prefix(0, torch.randn(33, hidden + 2 * kv, generator=gen(5), device="cuda").bfloat16())
        return a, DecodeStep(hidden, kv, vocab, slots, 16, n, attend=a)
    (a, eager), (b, captured) = make(), make()
    x, residual = (torch.randn(n, hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    slot = torch.randint(-1, slots, (n,), generator=g, device="cuda").int()
    tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda").int()
    captured(x, residual, slot, tokens)
    b.lens.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = captured(x, residual, slot, tokens)
    for i in range(5):
        x.normal_(generator=g)
        tokens.random_(0, vocab, generator=g)
        graph.replay()
        want = eager(x, residual, slot, tokens)
        torch.cuda.synchronize()
        assert a.lens.tolist() == b.lens.tolist() == [i + 1] * n
        assert torch.equal(held.attended, want.attended) and torch.equal(held.logits, want.logits)
        assert torch.equal(held.scores.logprob, want.scores.logprob)


def test_a_part_of_the_rows_and_a_full_cache():
    g = gen(4)
    a = CachedAttention(HEADS, KV, DIM, 6, 3, (20, 5, 9))
    for _ in range(5):
        qkv = torch.randn(4, (HEADS + 2 * KV) * DIM, generator=g, device="cuda").bfloat16()
        assert torch.isfinite(a(qkv)).all()
    assert a.lens.tolist() == [3] * 4 + [0] * 2


def test_the_command():
    r = subprocess.run([sys.executable, "-m", "tenant_lora_serving_amd.decode_step", "--rows", "3", "--adapters", "2",
                        "--context", "100", "--prefix", "50"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "us a step" in r.stdout, r.stderr[-2000:]
