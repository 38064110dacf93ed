"""The serving-step operators (norm, shared projection with adapters, token
log probabilities) against their definitions in 64 bits, on the GPU.

Tolerances: a rounding to a type is off by at most half a step, eps / 2 of the
value (bf16 2^-8, e4m3 2^-4 and half its smallest step 2^-10), and sums of fp32
products by a few units of 2^-24 of the sum of their absolute values."""
import math

import pytest
import torch

from tenant_lora_serving_amd import lora as B
from tenant_lora_serving_amd import step

pytestmark = pytest.mark.gpu

EPS = 1e-5
BF16, E4M3, U = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def padded(t, pad):
    """The same rows in a buffer with `pad` more columns, which hold NaN."""
    if not pad:
        return t
    raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    wide = torch.full((t.shape[0], t.shape[1] + pad), 0x7f if raw.dtype == torch.uint8 else math.nan,
                      dtype=raw.dtype, device=t.device)
    wide[:, :t.shape[1]] = raw
    return wide[:, :t.shape[1]].view(t.dtype)


def within(got, want, tol, what):
    got, want, tol = got.double(), want.double(), tol.double()
    bad = ~((got - want).abs() <= tol)
    bad &= ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {want[bad][0]}")


# ---------------------------------------------------------------- norm
def norm64(x, residual, w):
    s = x.double() if residual is None else x.double() + residual.double()
    y = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + EPS) * w.double()
    return s, y, y.abs().amax(dim=1) / 448.0


def check_norm(x, residual, w, bf16, quant, r):
    s, y, scale = norm64(x, residual, w)
    h = x.shape[1]
    rel = (h / 64 + 32) * U     # a thread's chain of squares, its tree, and the elementwise roundings
    if bf16:
        within(r.y, y, y.abs() * (BF16 + 2 * rel) + 1e-38, "y")
    else:
        assert r.y is None
    if residual is not None:
        within(r.residual, s, s.abs() * (BF16 + U) + 1e-38, "residual")
    else:
        assert r.residual is None
    if quant:
        within(r.q_scale, scale, scale * 2 * rel + 1e-44, "q_scale")
        live = scale > 0
        q = torch.where(live[:, None], y / torch.where(live, scale, 1.0)[:, None], 0.0)
        within(r.q.float(), q, q.abs() * (E4M3 + 4 * rel) + 2.0 ** -10 * (1 + 4 * rel), "q")
    else:
        assert r.q is None and r.q_scale is None


@pytest.mark.parametrize("n,h", [(1, 8), (1, 4096), (3, 64), (5, 512), (7, 520), (4, 1024), (9, 1032), (2, 2048),
                                 (3, 2056), (2, 4104), (3, 8192), (2, 8200), (2, 16384), (1, 16392), (2, 32768),
                                 (300, 4096), (1021, 136)])
@pytest.mark.parametrize("residual,bf16,quant,pad", [(True, True, True, 0), (False, True, False, 8),
                                                     (True, False, True, 136)])
def test_norm(n, h, residual, bf16, quant, pad):
    print(f"norm n={n} h={h} residual={residual} bf16={bf16} quant={quant} pad={pad}", flush=True)
    g = gen(n * 100003 + h)
    x = padded(randn(g, n, h).bfloat16(), pad)
    res = padded(randn(g, n, h, std=2.0).bfloat16(), pad) if residual else None
    w = (1 + randn(g, h, std=0.1)).bfloat16()
    r = step.rms_norm(x, w, EPS, residual=res, bf16=bf16, quant=quant)
    check_norm(x, res, w, bf16, quant, r)


def test_norm_in_place_residual():
    g = gen(3)
    x, res, w = randn(g, 6, 4096).bfloat16(), randn(g, 6, 4096).bfloat16(), (1 + randn(g, 4096)).bfloat16()
    keep = res.clone()
    r = step.rms_norm(x, w, EPS, residual=res, quant=True, residual_out=res)
    assert r.residual is res
    check_norm(x, keep, w, True, True, r)


def test_norm_of_zero_tiny_and_broken_rows():
    h = 1536
    x = randn(gen(4), 6, h)
    x[0] = 0
    x[1] *= 1e-30
    x[2, 7] = math.inf
    x[3, 100] = math.nan
    x[4] *= 1e25          # squares past fp32
    x = x.bfloat16()
    w = torch.ones(h, device="cuda").bfloat16()
    r = step.rms_norm(x, w, EPS, quant=True)
    check_norm(x[[0, 1, 5]], None, w, True, True, step.NormResult(r.y[[0, 1, 5]], None, r.q.float()[[0, 1, 5]],
                                                                   r.q_scale[[0, 1, 5]]))
    assert r.q_scale[0] == 0 and (r.q.float()[0] == 0).all()
    assert r.q_scale[2:4].isnan().all() and (r.q.float()[2:4] == 0).all()
    assert r.y[2, 7].isnan() and r.y[3].isnan().all()
    assert (r.y[4] == 0).all() and r.q_scale[4] == 0 and (r.q.float()[4] == 0).all()


def test_norm_of_a_row_whose_values_are_denormal_in_8_bits_scale():
    # the largest |y| is far below 448 / the largest float: its reciprocal scale would overflow
    h = 64
    x = torch.ones(1, h, device="cuda").bfloat16()
    w = torch.full((h,), 2.0 ** -126, device="cuda").bfloat16()
    w[1] = 2.0 ** -127
    r = step.rms_norm(x, w, 0.0, quant=True)
    assert r.q.float()[0, 0] == 448 and r.q.float()[0, 1] == 224


# ---------------------------------------------------------------- projection
def linear_inputs(seed, n, k, widths, S, R, fp8=False, pad=0, slot=None, bare=0.1):
    g = gen(seed)
    N, L = sum(widths), len(widths)
    x, w = randn(g, n, k), randn(g, N, k, std=k ** -0.5)
    a = randn(g, S, L, R, k, std=k ** -0.5).bfloat16()
    b = randn(g, S, N, R, std=R ** -0.5).bfloat16()
    scale = 0.25 + torch.rand(S, generator=g, device="cuda")
    if slot is None:
        slot = torch.randint(0, S, (n,), generator=g, device="cuda")
        slot = torch.where(torch.rand(n, generator=g, device="cuda") < bare, -1, slot)
    kw = {}
    if fp8:
        xs, ws = (t.abs().amax(dim=1).clamp_min(1e-12) / 448 for t in (x, w))
        kw = dict(xq=padded((x / xs[:, None]).to(torch.float8_e4m3fn), 2 * pad), x_scale=xs, w_scale=ws)
        w = (w / ws[:, None]).to(torch.float8_e4m3fn)
    else:
        w = w.bfloat16()
    return (padded(x.bfloat16(), pad), w, a, b, scale, widths, slot.to(torch.int32)), kw


def linear64(args, kw):
    """(values, a bound on their error) in 64 bits."""
    x, w, a, b, scale, widths, slot = args
    S, k = a.shape[0], x.shape[1]
    if kw:
        left, right = kw["xq"].double() * kw["x_scale"].double()[:, None], w.double() * kw["w_scale"].double()[:, None]
    else:
        left, right = x.double(), w.double()
    y, size = left @ right.T, left.abs() @ right.abs().T
    inner = torch.zeros_like(y)
    for s in range(S):
        rows = (slot == s).nonzero()[:, 0]
        lo = 0
        for l, width in enumerate(widths):
            if rows.numel():
                A, Bs = a[s, l].double(), b[s, lo:lo + width].double()
                y[rows, lo:lo + width] += scale[s].double() * (x[rows].double() @ A.T) @ Bs.T
                size[rows, lo:lo + width] += scale[s].double() * (x[rows].double().abs() @ A.abs().T) @ Bs.abs().T
                inner[rows, lo:lo + width] = scale[s].double() * (x[rows].double() @ A.T).abs() @ Bs.abs().T
            lo += width
    # one rounding to bf16; fp32 sums (k terms, in at least four chains); the
    # inner sums as two bf16 terms
    return y, y.abs() * BF16 + size * (k / 4 + 64) * U + inner * 2.0 ** -16


def check_linear(args, kw, got, what):
    y, tol = linear64(args, kw)
    within(got, y, tol, what)


SHAPES = [
    # n, k, widths, S, R
    (1, 16, (8,), 1, 8), (1, 4096, (512, 128, 128), 32, 16), (5, 48, (16,), 2, 24), (16, 64, (64,), 4, 8),
    (17, 128, (72, 8), 3, 16), (37, 1040, (200,), 8, 8), (63, 272, (8, 24, 40), 64, 128), (64, 512, (128,), 64, 64),
    (65, 256, (136,), 7, 32), (100, 2064, (96, 32), 9, 16), (256, 1024, (384, 128, 128), 32, 16),
    (257, 80, (264,), 5, 128), (300, 320, (256, 256), 300, 8), (520, 192, (328, 56), 64, 24),
    (1025, 144, (120,), 16, 64), (1500, 512, (512, 264), 16, 64), (2300, 1024, (776, 512), 3, 16),
    (2049, 400, (1032,), 64, 128),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k,widths,S,R", SHAPES)
def test_linear(n, k, widths, S, R, fp8):
    print(f"linear n={n} k={k} widths={widths} S={S} R={R} fp8={fp8}", flush=True)
    args, kw = linear_inputs(n + k, n, k, widths, S, R, fp8, pad=8 if n % 2 else 0)
    check_linear(args, kw, step.lora_linear(*args, **kw), "linear")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 70, 700, 2500])
@pytest.mark.parametrize("kind", ["none", "one", "runs", "invalid"])
def test_linear_slots(n, kind, fp8):
    print(f"linear slots n={n} kind={kind} fp8={fp8}", flush=True)
    S = 6
    at = torch.arange(n, device="cuda")
    slot = {"none": torch.full_like(at, -1), "one": torch.full_like(at, 4), "runs": at * 5 // n,
            "invalid": torch.where(at % 3 == 0, S + at, at % S)}[kind]
    args, kw = linear_inputs(n, n, 384, (264, 120), S, 16, fp8, slot=slot)
    check_linear(args, kw, step.lora_linear(*args, **kw), kind)


@pytest.mark.parametrize("n", [40, 2100])
def test_linear_out_and_workspace_of_a_larger_call(n):
    big, kwb = linear_inputs(1, 2500, 512, (512,), 64, 64)
    ws = step.linear_workspace(2500, 512, 512, 1, 64)
    step.lora_linear(*big, ws=ws)
    args, kw = linear_inputs(2, n, 256, (136, 64), 5, 16)
    wide = torch.full((n, 264), 7.0, device="cuda").bfloat16()
    for _ in range(2):
        got = step.lora_linear(*args, out=wide[:, :200], ws=ws)
        check_linear(args, kw, got, "out")
        assert (wide[:, 200:] == 7).all()
    check_linear(big, kwb, step.lora_linear(*big, ws=ws), "larger call again")


@pytest.mark.parametrize("n", [50, 2500])
def test_linear_other_stream_and_graph(n):
    args, kw = linear_inputs(9, n, 256, (136, 64), 5, 16)
    want = step.lora_linear(*args)
    check_linear(args, kw, want, "eager")
    ws = step.linear_workspace(n, 256, 200, 2, 16)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step.lora_linear(*args, out=out, ws=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.lora_linear(*args, out=out, ws=ws)
    for i in range(3):
        args[0].copy_(randn(gen(20 + i), n, 256).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step.lora_linear(*args))


# ---------------------------------------------------------------- log probabilities
def check_score(logits, tokens, top, r):
    z, t = logits.double(), tokens.long()
    n, v = z.shape
    logp = torch.where(z == -math.inf, z, torch.log_softmax(z, dim=1))
    given = (t >= 0) & (t < v)
    at = t.clamp(0, v - 1)[:, None]
    want = torch.where(given, logp.gather(1, at)[:, 0], 0.0)
    want = torch.where(t >= v, math.nan, want)
    # the distance to the maximum and the sum's logarithm, a few roundings each
    within(r.logprob, want, 4e-6 + want.abs().nan_to_num(0, 0, 0) * 4 * U, "logprob")
    rank = torch.where(given, 1 + (z > z.gather(1, at)).sum(dim=1), 0)
    assert torch.equal(r.rank.long(), rank)
    entropy = torch.special.entr(logp.exp()).sum(dim=1)
    within(r.entropy, entropy, 4e-6 + entropy.abs() * 64 * U, "entropy")
    if top == 0:
        assert r.top_ids is None and r.top_logprobs is None
        return
    order = torch.sort(z.cpu(), dim=1, descending=True, stable=True).indices[:, :top].to(z.device)
    best = logp.gather(1, order)
    if order.shape[1] < top:
        order = torch.nn.functional.pad(order, (0, top - order.shape[1]))
        best = torch.nn.functional.pad(best, (0, top - best.shape[1]), value=-math.inf)
    ids = torch.where(best > -math.inf, order, -1)
    assert torch.equal(r.top_ids.long(), ids)
    within(r.top_logprobs, best, 4e-6 + best.abs().nan_to_num(0, 0, 0) * 4 * U, "top_logprobs")


def tokens_for(g, n, v):
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    t[::5] = -1
    return t.to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
@pytest.mark.parametrize("n,v,pad", [(1, 1, 0), (2, 3, 1), (3, 7, 0), (1, 17, 0), (5, 500, 1), (1, 4097, 0),
                                     (2, 32003, 5), (1, 128256, 0), (3, 262144, 0), (600, 999, 0), (520, 33000, 56)])
def test_score(n, v, pad, top, dtype):
    print(f"score n={n} v={v} pad={pad} top={top} {dtype}", flush=True)
    g = gen(n + v)
    z = padded((randn(g, n, v, std=3.0)).to(dtype), pad)
    t = tokens_for(g, n, v)
    check_score(z, t, top, step.token_logprobs(z, t, top))


def odd_rows(kind, v, g):
    z = randn(g, 4, v, std=2.0)
    if kind == "masked":                 # rows with nothing, one, few and most masked
        z[0] = -math.inf
        z[1] = torch.where(torch.arange(v, device="cuda") == v // 2, z[1], -math.inf)
        z[2] = torch.where(torch.arange(v, device="cuda") % 97 == 5, z[2], -math.inf)
        z[3] = torch.where(torch.rand(v, generator=g, device="cuda") < 0.99, -math.inf, z[3])
    elif kind == "equal":                # nothing but ties
        z[0], z[1] = 0.0, -5.0
        z[2] = torch.where(torch.arange(v, device="cuda") % 2 == 0, 0.0, -0.0)
        z[3] = torch.randint(0, 2, (v,), generator=g, device="cuda").float()
    elif kind == "lowest":               # a mask of the type's lowest value
        low = torch.finfo(torch.bfloat16).min
        z[0] = low
        z[1, : v - 1] = low
        z[2, ::2] = low
        z[3, 1:] = low
    elif kind == "sorted":               # the largest at the end, at the start, in one thread's vectors
        z = z.sort(dim=1).values
        z[1] = z[1].flip(0)
        z[2, : min(v, 8)] += 50
        z[3, -min(v, 40):] += 50
    elif kind == "peaked":
        z[:, v // 3] = 200.0
        z[1] *= 1e4
        z[2] *= 1e-4
    return z


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["masked", "equal", "lowest", "sorted", "peaked"])
@pytest.mark.parametrize("v,top", [(40, 32), (5000, 20), (40007, 32), (128256, 1)])
def test_score_odd_rows(v, top, kind, dtype):
    print(f"score odd v={v} top={top} kind={kind} {dtype}", flush=True)
    g = gen(v)
    z = odd_rows(kind, v, g).to(dtype)
    t = torch.tensor([v // 2, v // 3, 0, v - 1], dtype=torch.int32, device="cuda")
    many = z.repeat(150, 1)              # a row's parts by one workgroup, or by fewer
    check_score(z, t, top, step.token_logprobs(z, t, top))
    if v <= 5000:
        check_score(many, t.repeat(150), top, step.token_logprobs(many, t.repeat(150), top))


def test_score_broken_rows_and_tokens():
    v = 3000
    z = randn(gen(8), 5, v)
    z[0, 17] = math.nan
    z[1, 18] = math.inf
    t = torch.tensor([5, 6, v, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    r = step.token_logprobs(z, t, 4)
    assert r.logprob[:2].isnan().all() and r.entropy[:2].isnan().all()
    assert ((r.top_ids >= -1) & (r.top_ids < v)).all()
    check_score(z[2:], t[2:], 4, step.LogprobResult(*(f[2:] for f in r)))


def test_score_workspace_between_shapes_and_graph():
    ws = step.logprobs_workspace(64, 40000, 32)
    for n, v, top in [(2, 30000, 20), (64, 40000, 32), (1, 9000, 0), (3, 20000, 5), (2, 30000, 20)]:
        g = gen(n * v)
        z, t = randn(g, n, v, std=3.0), tokens_for(g, n, v)
        check_score(z, t, top, step.token_logprobs(z, t, top, ws=ws))
    z, t = randn(gen(1), 4, 20000).bfloat16(), tokens_for(gen(2), 4, 20000)
    step.token_logprobs(z, t, 5, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step.token_logprobs(z, t, 5, ws=ws)
    for i in range(3):
        z.copy_(randn(gen(30 + i), 4, 20000, std=3.0).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        check_score(z, t, 5, r)


# ---------------------------------------------------------------- refusals, no rows
def test_calls_without_rows():
    args, kw = linear_inputs(1, 0, 64, (16,), 2, 8)
    assert step.lora_linear(*args).shape == (0, 16)
    z = torch.empty(0, 100, device="cuda")
    assert step.token_logprobs(z, torch.empty(0, dtype=torch.int32, device="cuda"), 3).top_ids.shape == (0, 3)
    x = torch.empty(0, 64, device="cuda").bfloat16()
    assert step.rms_norm(x, torch.ones(64, device="cuda").bfloat16(), quant=True).q.shape == (0, 64)


def test_refusals():
    x = torch.zeros(4, 64, device="cuda").bfloat16()
    w = torch.zeros(64, device="cuda").bfloat16()
    with pytest.raises(TypeError):
        step.rms_norm(x.float(), w)
    with pytest.raises(ValueError):
        step.rms_norm(x, w[:32])
    with pytest.raises(B.LoraError):
        step.rms_norm(x[:, :60].contiguous(), w[:60].contiguous())
    with pytest.raises(B.LoraError):
        step.rms_norm(x, w, bf16=False)
    with pytest.raises(ValueError):
        step.rms_norm(x.t(), w)
    args, kw = linear_inputs(1, 4, 64, (16,), 2, 8, fp8=True)
    with pytest.raises(TypeError):
        step.lora_linear(*args)                      # 8-bit weights without xq
    with pytest.raises(ValueError):
        step.lora_linear(*args, xq=kw["xq"])
    with pytest.raises(ValueError):
        step.lora_linear(*args[:5], (8,), args[6], **kw)
    with pytest.raises(B.LoraError) as e:
        step.lora_linear(*args, **kw, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -3
    z = torch.zeros(2, 100, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(B.LoraError) as e:
        step.token_logprobs(z, t, 33)
    assert e.value.status == -2
    with pytest.raises(TypeError):
        step.token_logprobs(z, t.long())
    with pytest.raises(TypeError):
        step.token_logprobs(z.half(), t)


# ---------------------------------------------------------------- projection: broken adapters, more paths
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [3, 30, 200, 700, 2100])
def test_linear_broken_adapter_stays_with_its_rows(n, fp8):
    """An infinity or NaN in one row, or in one tenant's adapter, shows in the
    results that it belongs to and in no other row's (from an inner sum it may
    reach the row's other columns, from B no other column)."""
    print(f"linear broken n={n} fp8={fp8}", flush=True)
    widths, k = (264, 120), 384
    args, kw = linear_inputs(n, n, k, widths, 5, 16, fp8, slot=torch.arange(n, device="cuda") % 5)
    x, w, a, b, scale, _, slot = args
    clean = linear64(args, kw)
    broken = torch.zeros(n, sum(widths), dtype=torch.bool, device="cuda")
    x, a, b = x.clone(), a.clone(), b.clone()
    x[1, 5] = math.inf                  # a row of slot 1
    broken[1] = True
    b[2, 7, 3], b[2, 300, 0] = math.nan, math.inf
    broken[(slot == 2)[:, None] & (torch.arange(sum(widths), device="cuda") == 7)[None, :]] = True
    broken[(slot == 2)[:, None] & (torch.arange(sum(widths), device="cuda") == 300)[None, :]] = True
    a[3, 1, 2] = math.nan               # one of the second slice's inner sums
    broken[(slot == 3)[:, None] & (torch.arange(sum(widths), device="cuda") >= 264)[None, :]] = True
    got = step.lora_linear(x, w, a, b, scale, widths, slot, **kw)
    assert not got[broken].isfinite().any()
    y, tol = clean
    rest = ~broken & (slot != 3)[:, None]
    within(got[rest], y[rest], tol[rest], "the others")


@pytest.mark.parametrize("n", [2, 100, 700, 1200])
def test_linear_inner_sums_past_the_largest_bf16(n):
    # 3.397e38 is finite in fp32 and rounds to infinity in bf16
    k = 272
    x = torch.zeros(n, k, device="cuda")
    x[:, 0], x[:, 1] = 3.38953139e38, 7.5e35
    a, b = torch.ones(1, 1, 8, k, device="cuda"), torch.full((1, 16, 8), 2.0 ** -100, device="cuda")
    args = (x.bfloat16(), torch.zeros(16, k, device="cuda").bfloat16(), a.bfloat16(), b.bfloat16(),
            torch.ones(1, device="cuda"), (16,), torch.zeros(n, dtype=torch.int32, device="cuda"))
    check_linear(args, {}, step.lora_linear(*args), "large inner sums")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k,widths,S,R", [
    (33, 336, (16,), 40, 8), (511, 512, (136, 80), 512, 16), (512, 2064, (392,), 1, 24), (513, 64, (520, 8), 70, 128),
    (640, 4096, (640, 128, 128), 32, 16), (900, 1536, (2056,), 6, 64), (1024, 272, (64, 64), 1024, 8),
    (1100, 256, (512, 40), 9, 32), (1300, 16, (8,), 2, 8), (1800, 640, (72,), 16, 16), (5000, 96, (48,), 5000, 8),
])
def test_linear_more_shapes(n, k, widths, S, R, fp8):
    print(f"linear n={n} k={k} widths={widths} S={S} R={R} fp8={fp8}", flush=True)
    args, kw = linear_inputs(n + k, n, k, widths, S, R, fp8, pad=16 if n % 2 else 0)
    check_linear(args, kw, step.lora_linear(*args, **kw), "linear")


def test_one_workspace_through_every_path():
    ws = step.linear_workspace(3000, 512, 512, 2, 64)
    for n, k, widths, S, R in [(3000, 512, (264, 248), 9, 64), (4, 512, (64,), 3, 16), (700, 384, (72,), 30, 8),
                               (4, 512, (64,), 3, 16), (300, 48, (16, 16), 7, 64), (3000, 512, (264, 248), 9, 64)]:
        args, kw = linear_inputs(n, n, k, widths, S, R)
        for _ in range(2):
            check_linear(args, kw, step.lora_linear(*args, ws=ws), f"n={n}")


def test_calls_on_another_stream_allocate_there():
    side = torch.cuda.Stream()
    args, kw = linear_inputs(9, 50, 256, (136, 64), 5, 16)
    z, t = randn(gen(1), 4, 20000), tokens_for(gen(2), 4, 20000)
    x, w = randn(gen(3), 6, 512).bfloat16(), torch.ones(512, device="cuda").bfloat16()
    side.wait_stream(torch.cuda.current_stream())
    y = step.lora_linear(*args, stream=side)
    r = step.token_logprobs(z, t, 5, stream=side)
    q = step.rms_norm(x, w, EPS, quant=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_linear(args, kw, y, "side stream")
    check_score(z, t, 5, r)
    check_norm(x, None, w, True, True, q)


@pytest.mark.parametrize("n", [20, 700])
def test_linear_graph_replays(n):
    args, kw = linear_inputs(5, n, 512, (136, 64), 6, 16)
    ws = step.linear_workspace(n, 512, 200, 2, 16)
    out = step.lora_linear(*args, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.lora_linear(*args, out=out, ws=ws)
        step.lora_linear(*args, out=out, ws=ws)
    for i in range(4):
        args[0].copy_(randn(gen(40 + i), n, 512).bfloat16())
        args[6].copy_(torch.randint(-1, 6, (n,), generator=gen(50 + i), device="cuda").int())
        graph.replay()
        torch.cuda.synchronize()
        check_linear(args, kw, out, f"replay {i}")
        assert torch.equal(out, step.lora_linear(*args, ws=ws))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k,widths,S,R", [
    (1000, 2064, (2000, 1008), 20, 24), (700, 1040, (4104,), 700, 8), (257, 4096, (8, 8184), 3, 128),
    (513, 528, (7176, 1000), 40, 16), (900, 1552, (1536, 1536, 1528), 2, 64), (384, 272, (16392,), 5, 32),
])
def test_linear_middling(n, k, widths, S, R, fp8):
    print(f"linear middling n={n} k={k} widths={widths} S={S} R={R} fp8={fp8}", flush=True)
    args, kw = linear_inputs(n + k, n, k, widths, S, R, fp8, pad=16 if n % 2 else 0)
    check_linear(args, kw, step.lora_linear(*args, **kw), "linear")


@pytest.mark.parametrize("fp8", [False, True])
def test_linear_middling_broken_adapter(fp8):
    n, widths, k = 600, (4000, 2008), 1040
    args, kw = linear_inputs(3, n, k, widths, 7, 16, fp8, slot=torch.arange(n, device="cuda") % 7)
    x, w, a, b, scale, _, slot = args
    y, tol = linear64(args, kw)
    b = b.clone()
    b[2, 7, 3], b[4, 5000, 0] = math.nan, math.inf
    at = torch.arange(sum(widths), device="cuda")[None, :]
    broken = (slot == 2)[:, None] & (at == 7) | (slot == 4)[:, None] & (at == 5000)
    got = step.lora_linear(x, w, a, b, scale, widths, slot, **kw)
    assert not got[broken].isfinite().any()
    within(got[~broken], y[~broken], tol[~broken], "the others")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,k,widths,S,R", [(200, 272, (16392,), 50, 16), (100, 528, (20008, 6000), 9, 24),
                                            (65, 80, (24584,), 65, 8), (256, 4096, (12296,), 4, 64)])
def test_linear_few_rows_by_many_columns(n, k, widths, S, R, fp8):
    print(f"linear wide n={n} k={k} widths={widths} S={S} R={R} fp8={fp8}", flush=True)
    args, kw = linear_inputs(n + k, n, k, widths, S, R, fp8)
    check_linear(args, kw, step.lora_linear(*args, **kw), "linear")


def test_norm_of_more_rows_than_one_side_of_a_grid():
    n, h = (1 << 22) + 5, 8         # four rows a workgroup, 2^20 workgroups a side
    x = randn(gen(6), n, h).bfloat16()
    w = (1 + randn(gen(7), h, std=0.1)).bfloat16()
    check_norm(x, None, w, True, True, step.rms_norm(x, w, EPS, quant=True))
