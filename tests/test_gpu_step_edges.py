"""The serving-step operators at the edges of what they accept, against their
definitions in 64 bits, on the GPU (tolerances as in test_gpu_step.py)."""
import pytest

from tenant_lora_serving_amd import step
from tenant_lora_serving_amd.decode_step import DecodeStep
from test_gpu_decode_step import inputs
from test_gpu_step import check_linear, check_score, gen, randn, tokens_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,vocab", [(128, 128256), (512, 32000)])
def test_decode_step_of_fewer_rows_than_it_was_made_for(most, vocab):
    run = DecodeStep(256, 64, vocab, 4, 8, most)
    for n in (1, 5, 100, 127, most - 1, most):
        print(f"decode step of {n} rows, made for {most}, vocabulary {vocab}", flush=True)
        args = inputs(n, n, 256, vocab, 4)
        r = run(*args)
        p = run.head
        check_linear((r.final.y, p.w, p.a_pool, p.b_pool, run.scale, p.sizes, args[2]), {}, r.logits, "head")
        check_score(r.logits, args[3], run.top, r.scores)


@pytest.mark.parametrize("v", [4100, 32000, 70000])
def test_score_workspace_of_a_larger_batch(v):
    ws = step.logprobs_workspace(600, v, 8)
    for n, top in ((600, 8), (1, 8), (37, 3), (255, 8), (511, 0), (512, 8)):
        print(f"score n={n} v={v} top={top}", flush=True)
        z, t = randn(gen(n + v), n, v, std=3.0).bfloat16(), tokens_for(gen(n), n, v)
        check_score(z, t, top, step.token_logprobs(z, t, top, ws=ws))
