"""The serving-step operators run together: every stage of the example's step
against its 64-bit definition on that stage's own inputs, and as a graph."""
import pytest
import torch

from tenant_lora_serving_amd.decode_step import EPS, DecodeStep
from test_gpu_step import check_linear, check_norm, check_score, gen, randn

pytestmark = pytest.mark.gpu
assert EPS == 1e-5   # (check_norm's)


def inputs(seed, n, hidden, vocab, slots):
    g = gen(seed)
    return (randn(g, n, hidden).bfloat16(), randn(g, n, hidden).bfloat16(),
            torch.randint(-1, slots, (n,), generator=g, device="cuda").int(),
            torch.randint(-1, vocab, (n,), generator=g, device="cuda").int())


@pytest.mark.parametrize("n", [1, 37, 300])
def test_stages_and_graph(n):
    hidden, kv, vocab, slots = 512, 128, 5000, 6
    run = DecodeStep(hidden, kv, vocab, slots, 16, n)
    args = inputs(n, n, hidden, vocab, slots)
    x, residual, slot, tokens = args
    r = run(*args)
    check_norm(x, residual, run.norms[0], True, True, r.norm)
    p = run.qkv
    check_linear((r.norm.y, p.w, p.a_pool, p.b_pool, run.scale, p.sizes, slot),
                 dict(xq=r.norm.q, x_scale=r.norm.q_scale, w_scale=p.w_scale), r.qkv, "qkv")
    p = run.o
    check_linear((r.attended, p.w, p.a_pool, p.b_pool, run.scale, p.sizes, slot), {}, r.o, "o")
    check_norm(r.o, r.norm.residual, run.norms[1], True, False, r.final)
    p = run.head
    check_linear((r.final.y, p.w, p.a_pool, p.b_pool, run.scale, p.sizes, slot), {}, r.logits, "head")
    check_score(r.logits, tokens, run.top, r.scores)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(*args)
    for i in range(3):
        for t, new in zip(args, inputs(100 + i, n, hidden, vocab, slots)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        again = run(*args)
        assert torch.equal(held.logits, again.logits)
        assert torch.equal(held.scores.logprob, again.scores.logprob)
        assert torch.equal(held.scores.top_ids, again.scores.top_ids)
