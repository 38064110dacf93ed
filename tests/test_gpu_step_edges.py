"""The serving-step operators at the edges of what they accept, against their
definitions in 64 bits, on the GPU (tolerances as in test_gpu_step.py)."""
import math

import pytest
import torch

from tenant_lora_serving_amd import step
from tenant_lora_serving_amd.lora import LoraError
from tenant_lora_serving_amd.decode_step import DecodeStep
from test_gpu_decode_step import inputs
from test_gpu_step import BF16, E4M3, U, check_linear, check_score, gen, linear64, linear_inputs, randn, tokens_for, within

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


# ---------------------------------------------------------------- norm
def norm_definition(x, residual, w, eps):
    """y and the 8-bit copy's scale in 64 bits; a row of zeros is zero."""
    s = x.double() if residual is None else x.double() + residual.double()
    length = torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps)
    y = torch.where(s.abs().amax(dim=1, keepdim=True) > 0, s / length * w.double(), 0.0)
    return y, y.abs().amax(dim=1) / 448


def check_norm_eps(x, residual, w, eps):
    y, scale = norm_definition(x, residual, w, eps)
    r = step.rms_norm(x, w, eps, residual=residual, quant=True)
    rel = (x.shape[1] / 64 + 32) * U
    within(r.y, y, y.abs() * (BF16 + 2 * rel) + 1e-38, "y")
    within(r.q_scale, scale, scale * 2 * rel + 1e-44, "q_scale")
    live = scale > 0
    q = torch.where(live[:, None], y / torch.where(live, scale, 1.0)[:, None], 0.0)
    within(r.q.float(), q, q.abs() * (E4M3 + 4 * rel) + 2.0 ** -10 * (1 + 4 * rel), "q")
    return r


@pytest.mark.parametrize("h", [8, 1000, 4096, 20000])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 1e-36, 1e-30, 1e-5])
def test_norm_of_zero_and_tiny_rows_with_any_eps(eps, residual, h):
    print(f"norm tiny eps={eps} residual={residual} h={h}", flush=True)
    x = randn(gen(h), 9, h)
    for row, power in enumerate((0, -14, -48, -52, -70, -110, -124)):
        x[row] *= 2.0 ** power
    x = x.bfloat16()
    x[7] = 0
    x[8] = 0
    x[8, h // 2] = 2.0 ** -133           # the smallest bf16
    res = None
    if residual:
        res = x.flip(1).contiguous()
        res[7] = 0
    w = (1 + randn(gen(1), h, std=0.1)).bfloat16()
    r = check_norm_eps(x, res, w, eps)
    assert (r.y[7] == 0).all() and r.q_scale[7] == 0 and (r.q.float()[7] == 0).all()


@pytest.mark.parametrize("h", [64, 1000, 4096, 20000])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_norm_of_a_weight_that_is_not_finite(bad, h):
    print(f"norm weight {bad} h={h}", flush=True)
    x, w = randn(gen(h), 6, h).bfloat16(), (1 + randn(gen(1), h, std=0.1)).bfloat16()
    x[3] = 0
    x[4, h - 3] = 0                      # 0 times the weight is NaN, whatever the weight
    clean, _ = norm_definition(x, None, w, 1e-5)
    w[h - 3] = bad
    r = step.rms_norm(x, w, 1e-5, quant=True)
    assert r.q_scale.isnan().all() and (r.q.float() == 0).all()
    at, rest = r.y[:, h - 3].double(), torch.arange(h, device="cuda") != h - 3
    assert not at.isfinite().any() and at[3:5].isnan().all()
    if not math.isnan(bad):
        assert torch.equal(at[:3], x[:3, h - 3].double() * bad)
    y = clean[:, rest]
    within(r.y[:, rest], y, y.abs() * (BF16 + 2 * (h / 64 + 32) * U) + 1e-38, "the other columns")


@pytest.mark.parametrize("h", [64, 4096, 20000])
def test_norm_of_rows_whose_products_with_the_weight_pass_fp32(h):
    x, w = (randn(gen(h), 4, h) * 1e15).bfloat16(), (1 + randn(gen(1), h, std=0.1)).bfloat16()
    w[5] = 1e30                          # x w is past fp32, y is not
    check_norm_eps(x, None, w, 1e-5)
    x[2] = 0
    check_norm_eps(x, None, w, 0.0)


@pytest.mark.parametrize("h", [64, 4096, 20000])
@pytest.mark.parametrize("power", [-60, -96, -110])
def test_norm_of_rows_whose_products_with_the_weight_vanish(power, h):
    # x w is below fp32's smallest numbers, y is not
    x = (randn(gen(h), 3, h) * 2.0 ** -45).bfloat16()
    w = ((1 + randn(gen(1), h, std=0.1)) * 2.0 ** power).bfloat16()
    check_norm_eps(x, None, w, 0.0)


# ---------------------------------------------------------------- sizes past 32 bits
def test_sizes_past_32_bits_are_refused():
    far = 1 << 32                        # (17 GB, never written)
    x = torch.empty(1, far + 64, dtype=torch.bfloat16, device="cuda")
    token = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: step.rms_norm(x, x[0], quant=True), lambda: step.token_logprobs(x, token, 2),
                 lambda: step.token_logprobs(x[:, :100], token, far + 2)):
        with pytest.raises(LoraError) as e:
            call()
        assert e.value.status == -2


# ---------------------------------------------------------------- the largest sizes and spans
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k,widths", [(4, 64, (72,)), (300, 64, (72,)), (2100, 272, (1992, 2000))])
def test_linear_rows_as_far_apart_as_the_limit(n, k, widths, fp8):
    print(f"linear span n={n} k={k} fp8={fp8}", flush=True)
    args, kw = linear_inputs(n, n, k, widths, 5, 16, fp8)
    x, rest = args[0], args[1:]
    want = step.lora_linear(*args, **kw)
    check_linear(args, kw, want, "close rows")

    def spread(t, ld):
        far = torch.zeros(n * ld, dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype, device="cuda")
        rows = far.as_strided((n, k), (ld, 1))
        rows.copy_(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t)
        return rows.view(t.dtype)
    ldx, ldxq = ((1 << 30) - 1) // n // 8 * 8, ((1 << 31) - 1) // n // 16 * 16
    assert torch.equal(step.lora_linear(spread(x, ldx), *rest, **kw), want)
    if fp8:
        kw = dict(kw, xq=spread(kw["xq"], ldxq))
        assert torch.equal(step.lora_linear(x, *rest, **kw), want)
    with pytest.raises(LoraError) as e:
        step.lora_linear(x.new_zeros((n, ldx + 8))[:, :k], *rest, **kw)
    assert e.value.status == -2


@pytest.mark.parametrize("n", [3, 100, 300, 3000])
def test_linear_most_slots(n):
    print(f"linear 8192 slots n={n}", flush=True)
    S = 8192
    slot = torch.randint(S - 64, S, (n,), generator=gen(n), device="cuda")
    slot[0], slot[1], slot[2] = S - 1, 0, S
    args, kw = linear_inputs(n, n, 64, (72, 8), S, 8, slot=torch.where(slot == S, S - 1, slot))
    check_linear(args, kw, step.lora_linear(*args), "linear")
    past = (*args[:6], slot.int())           # S is no slot
    check_linear(past, kw, step.lora_linear(*past), "linear")


def whole_numbers(seed, n, k, widths, S, R, fp8):
    """Small whole numbers, so that every sum is exact in fp32 and every result
    the rounding of a whole number, however long the sum."""
    g, N = gen(seed), sum(widths)

    def whole(most, *shape):
        return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8).bfloat16()
    x, w = whole(1, n, k), whole(2, N, k)
    slot = torch.randint(-1, S, (n,), generator=g, device="cuda").int()
    rest = (whole(1, S, len(widths), R, k), whole(1, S, N, R), torch.ones(S, device="cuda"), widths, slot)
    if not fp8:
        return (x, w, *rest), {}
    kw = dict(xq=x.to(torch.float8_e4m3fn), x_scale=torch.ones(n, device="cuda"), w_scale=torch.ones(N, device="cuda"))
    return (x, w.to(torch.float8_e4m3fn), *rest), kw


def check_whole(args, kw, got):
    y, _ = linear64(args, kw)
    assert y.abs().max() < 1 << 24 and torch.equal(got, y.float().bfloat16())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,widths", [(5, (16,)), (300, (200, 64)), (600, (1040,)), (2100, (3992,))])
def test_linear_longest_k(n, widths, fp8):
    print(f"linear longest k n={n} fp8={fp8}", flush=True)
    args, kw = whole_numbers(n, n, 1 << 18, widths, 2, 8, fp8)
    check_whole(args, kw, step.lora_linear(*args, **kw))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k,widths", [(3, 16, ((1 << 24) - 8, 8)), (1 << 18, 16, (8,)), (1 << 18, 272, (520,))])
def test_linear_most_columns_and_rows(n, k, widths, fp8):
    print(f"linear largest n={n} k={k} widths={widths} fp8={fp8}", flush=True)
    args, kw = whole_numbers(n, n, k, widths, 2, 8, fp8)
    check_whole(args, kw, step.lora_linear(*args, **kw))


@pytest.mark.parametrize("n,v,top", [(1 << 16, 64, 32), (1 << 16, 4200, 0), (2, 1 << 20, 32), (70, 1 << 20, 5)])
@pytest.mark.parametrize("fp32", [False, True])
def test_score_most_rows_and_logits(n, v, top, fp32):
    print(f"score largest n={n} v={v} top={top} fp32={fp32}", flush=True)
    z = randn(gen(n + v), n, v, std=3.0)
    z = z if fp32 else z.bfloat16()
    t = tokens_for(gen(n), n, v)
    check_score(z, t, top, step.token_logprobs(z, t, top))
