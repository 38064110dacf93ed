"""Calls of the paged cache's operators at the edge of what they accept: refusals, scales of 0 and not finite, and
the second, careful way of the many-row kernel in every form.  Definition and bounds are those of test_gpu_attend.py."""
import math

import pytest
import torch

from tenant_lora_serving_amd import step
from tenant_lora_serving_amd.decode_step import CachedAttention
from tenant_lora_serving_amd.lora import LoraError
from test_gpu_attend import Batch, check, gen, ints, near

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- tables
def test_tables_whose_rows_overlap_are_refused():
    b = Batch(70, [1] * 4, [40, 40, 40, 40], decode=True)
    for pages in (b.pages[:1].expand(4, -1), b.pages.as_strided((4, b.pages.shape[1]), (1, 1)), b.pages[:1, :1].expand(4, 1)):
        with pytest.raises(LoraError):
            b.call(pages=pages)
        with pytest.raises(LoraError):
            b.call(prefix=step.Prefixes(pages, b.len_t, ints([0, 1, 2, 3, 4])))
    # the same pages for every request, a row of memory each
    b.pages = b.pages[:1].repeat(4, 1)
    check(b, "one table")


# ---------------------------------------------------------------- scales of 0, infinite and NaN
def test_values_over_a_scale_of_0():
    """A 0 is stored as 0; other values over a scale of 0 are larger than 448 and stored as that; NaN stays."""
    x = torch.zeros(1, 2, 16, device="cuda", dtype=torch.bfloat16)
    x[0, :, :7] = torch.tensor([0.0, -0.0, 1.0, -1e-38, math.inf, -math.inf, math.nan], device="cuda")
    kc, vc = (torch.ones(1, 1, 2, 16, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    scale = torch.tensor([0.0, 1.0], device="cuda")
    step.kv_append(x, x, kc, vc, ints([0]), k_scale=scale, v_scale=scale)
    for c in (kc, vc):
        got = c.float()[0, 0]
        assert got[0, :6].tolist() == [0.0, 0.0, 448.0, -448.0, 448.0, -448.0] and math.isnan(got[0, 6].item())
        assert (got[0, 7:] == 0).all()
        assert got[1, :6].tolist() == [0.0, 0.0, 1.0, 0.0, 448.0, -448.0] and math.isnan(got[1, 6].item())


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("zero", ["head of zeros", "head of values"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_append_and_attend_with_a_scale_of_0(rows, zero, neighbours):
    """A head whose scale is 0 counts as zeros: its keys score 0, its values are 0."""
    n, kv, dim = 40, 2, 64
    g = gen(71)
    k, v = (torch.randn(n, kv, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(rows, 4, dim, generator=g, device="cuda").bfloat16()
    if zero == "head of zeros":
        k[:, 0], v[:, 1] = 0, 0
    kc, vc = (torch.zeros(3, 16, kv, dim, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    scales = dict(k_scale=torch.tensor([0.0, 0.01], device="cuda"), v_scale=torch.tensor([0.01, 0.0], device="cuda"))
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    step.kv_append(k, v, kc, vc, t, positions=t, rotation=step.rotation_table(n, dim), neighbours=neighbours, **scales)
    assert torch.isfinite(kc.float()).all() and torch.isfinite(vc.float()).all()
    r = step.paged_attention(q, kc, vc, ints([[0, 1, 2]]), ints([n]), starts=ints([0, rows]), max_rows=rows, causal=False,
                             lse=True, **scales)
    # the mean of the values in the cache: terms of p = 1, which bf16 holds, fp32 sums, one rounding
    held = vc.double().flatten(0, 1)[:n, 0] * scales["v_scale"][0].double()
    want, tol = held.mean(dim=0), held.mean(dim=0).abs() * 2.0 ** -8 + held.abs().sum(dim=0) * 2.0 ** -20
    near(r.out[:, :2], want.expand(rows, 2, dim), tol.expand(rows, 2, dim), "keys of scale 0")
    assert (r.out[:, 2:] == 0).all()
    # (p = 1 exactly: ln 40 from log2 and its product with ln 2)
    near(r.lse[:, :2], torch.full((rows, 2), math.log(n), dtype=torch.float64, device="cuda"),
         torch.full((rows, 2), 2.0 ** -20, dtype=torch.float64, device="cuda"), "lse")
    assert torch.isfinite(r.lse).all()


@pytest.mark.parametrize("rows,lens,prefixes", [
    ([1] * 5, [0, 40, 3000, 1, 300], ()), ([3, 2, 9, 1], [40, 0, 20, 1000], ()), ([40, 130, 7, 300], [300, 50, 0, 4000], ()),
    ([1] * 9, [0, 40, 0, 5, 70, 0, 9, 300, 1], ((50, 3), (0, 2))), ([20, 3, 50], [0, 300, 20], ((900, 2),))])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_scale_of_the_keys_that_is_not_finite(rows, lens, prefixes, value):
    """It reaches every row of its head that sees a key, and no other."""
    decode = max(rows) == 1
    b = Batch(72, rows, lens, cache="e4m3", prefixes=prefixes, first=0, decode=decode)
    out, lse, tol, tol_lse = b.want()
    b.k_scale[1] = value
    seen = torch.isfinite(lse[:, 4:])
    out[:, 4:][seen], lse[:, 4:][seen] = math.nan, math.nan
    assert seen.any() and not seen.all()
    check(b, f"scale {value}", want=(out, lse, tol, tol_lse))


# ---------------------------------------------------------------- the cached attention of a decode step
def test_lengths_that_lie_outside_the_cache():
    """A negative length counts as 0, one past the context as a full request: its last token is written over."""
    g = gen(73)
    a = CachedAttention(4, 2, 64, 3, 20)
    a.lens.copy_(ints([-5, 2 ** 31 - 1, -2 ** 31]))
    qkv = torch.randn(3, 8 * 64, generator=g, device="cuda").bfloat16()
    out = a(qkv).view(3, 4, 64)
    assert a.lens.tolist() == [1, 20, 1]
    v = a.parts(qkv)[2].repeat_interleave(2, dim=1)
    assert torch.equal(out[0], v[0]) and torch.equal(out[2], v[2])     # (a first token's own value)
    assert torch.isfinite(out[1]).all()


# ---------------------------------------------------------------- the careful way
def careful_batch(seed, rows, lens, prefixes, dim, cache, page):
    """Values that are not finite behind most of the rows, a NaN key that the last row alone sees, pages that are
    not there among the request's own and the prefix's: nothing of it may reach a row that does not see it."""
    b = Batch(seed, rows, lens, heads=4, kv=1, dim=dim, cache=cache, page=page, prefixes=prefixes)
    worst = math.nan if cache == "e4m3" else math.inf

    def at(table, j):
        return table[j // page].item(), j % page
    for request, (r, n) in enumerate(zip(rows, lens)):
        p, t = at(b.pages[request], n - 2)
        b.v_cache[p, t, 0, 7], b.v_cache[p, t, 0, dim - 1] = worst, math.nan
        if request == 0:
            p, t = at(b.pages[request], n - 1)
            b.k_cache[p, t, 0, 5], b.v_cache[p, t, 0, 3] = math.nan, -worst
    pages = b.pages.clone()
    pages[1, 0] = 2 ** 31 - 1
    if lens[0] // page // 2 < (lens[0] - 2) // page:
        pages[0, lens[0] // page // 2] = -1
    if prefixes:
        p, t = at(b.prefix.pages[1], prefixes[1][0] - 1)
        b.v_cache[p, t, 0, 9] = worst
        b.prefix.pages[0, 1] = b.k_cache.shape[0]
    return b, pages


@pytest.mark.parametrize("page", [3, 16, 100])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,lens", [([60, 9, 130], [60, 200, 300]), ([100, 33], [9000, 3000]), ([4, 3], [40, 130]),
                                       ([4, 2], [6000, 5000])])
@pytest.mark.parametrize("shared", [False, True])
def test_what_is_not_finite_reaches_no_row_before_it(page, dim, cache, rows, lens, shared):
    prefixes = ((2500, 1), (70, len(rows) - 1)) if shared else ()
    b, pages = careful_batch(80, rows, lens, prefixes, dim, cache, page)
    r = check(b, f"{dim} {cache} {page}", pages=pages)
    last = rows[0] - 1
    assert torch.isfinite(r.out[:last - 1]).all() and torch.isnan(r.out[last]).all()


def test_what_is_not_finite_reaches_every_row_that_sees_it():
    """A cut tile of which one piece is done the careful way, with the same bits each time."""
    rows, lens = [100, 33], [9000, 3000]
    b = Batch(81, rows, lens, heads=4, kv=1)
    b.v_cache[b.pages[0, 0].item(), 0, 0, 0] = math.inf      # (every row of request 0 sees it: its column 0 is infinite)
    r = check(b, "seen by all")
    assert torch.isinf(r.out[:100, :, 0]).all() and torch.isfinite(r.out[:, :, 1:]).all()
    again = b.call()
    assert torch.equal(r.out, again.out) and torch.equal(r.lse, again.lse)


def test_prefix_starts_that_make_no_sense_stay_inside():
    b = Batch(82, [1] * 9, [40] * 9, prefixes=((50, 4), (20, 3)), decode=True)
    c = Batch(83, [30] * 9, [40] * 9, prefixes=((50, 4), (20, 3)))
    for x in (b, c):
        n = x.q.shape[0]
        ws = step.attention_workspace(n, 8, 2, 128, prefixes=True)
        out = torch.full((n + 8, 8, 128), 7.0, device="cuda", dtype=torch.bfloat16)
        for ends in ([0, -5, 100], [9, 5, 1], [-1, -1, 2 ** 31 - 1], [2 ** 31 - 1, 0, -2 ** 31]):
            x.call(prefix=x.prefix._replace(starts=ints(ends)), out=out[4:-4], ws=ws)
            assert (out[:4] == 7).all() and (out[-4:] == 7).all()
        want = x.want()
        assert (ws[:4096] == 0).all()
        near(x.call(out=out[4:-4], ws=ws).out, want[0], want[2], "afterwards")
