"""Calls of the paged cache's operators at the edge of what they accept: refusals, scales of 0 and not finite, and
the second, careful way of the many-row kernel in every form.  Definition and bounds are those of test_gpu_attend.py."""
import copy
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


# ---------------------------------------------------------------- forms and sizes that no other test has
@pytest.mark.parametrize("rows", [[7, 0, 130, 1, 40], [2, 1, 0, 3, 2]])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
def test_prefixes_of_queries_to_another_sequence(rows, cache, dim):
    """Rows that all see every key of their prefix and their request, against a request of its own for each row."""
    lens = [40, 3, 900, 0, 129]
    b = Batch(90, rows, lens, dim=dim, cache=cache, prefixes=((300, 1), (70, 3)), first=1)
    each = copy.copy(b)
    of = [r for r, count in enumerate(rows) for _ in range(count)]
    each.rows, each.lens, each.pages = [1] * len(of), [lens[r] for r in of], b.pages[of].contiguous()
    each.first, each.prefixes = rows[0], ((300, rows[1]), (70, sum(rows[2:])))
    check(b, "not causal", causal=False, want=each.want())


def small_cache(g, pages, page, dim):
    return [torch.randn(pages, page, 1, dim, generator=g, device="cuda").bfloat16() for _ in range(2)]


def one_page(q, k, v, mask):
    """(out, bound) in 64 bits of rows that have keys k [rows, keys, dim] of their own; the bound as in test_gpu_attend.py,
    scores of 16 products of normal values being off by less than 2^-16."""
    q, k, v = q.double(), k.double()[:, None], v.double()[:, None]
    s = ((q[:, :, None] * k).sum(dim=3) * q.shape[2] ** -0.5).masked_fill(~mask[:, None], -math.inf)
    p = torch.where(mask[:, None], torch.softmax(s, dim=2), 0.0)[..., None]
    o = (p * v).sum(dim=2)
    return o, 2.0 ** -8 * o.abs() + (p * v.abs()).sum(dim=2) * (1.01 * 2.0 ** -8 + 2.0 ** -14)


def test_the_most_requests_and_prefixes():
    g, n, page, dim = gen(91), 1 << 16, 16, 16
    kc, vc = small_cache(g, 1000, page, dim)
    pages = torch.randint(0, 1000, (n, 1), generator=g, device="cuda").int()
    lens = torch.randint(0, page + 1, (n,), generator=g, device="cuda").int()
    q = torch.randn(n, 2, dim, generator=g, device="cuda").bfloat16()
    k, v = kc[pages[:, 0].long(), :, 0], vc[pages[:, 0].long(), :, 0]
    mask = torch.arange(page, device="cuda")[None] < lens[:, None]
    want = one_page(q, k, v, mask)
    near(step.paged_attention(q, kc, vc, pages, lens).out, *want, "tokens")
    each = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    near(step.paged_attention(q, kc, vc, pages, lens, starts=each, max_rows=200).out, *want, "the other kernel")
    prefix = step.Prefixes(pages.flip(0).contiguous(), lens.flip(0).contiguous(), each)
    want = one_page(q, *(torch.cat([x.flip(0), x], dim=1) for x in (k, v, mask)))
    near(step.paged_attention(q, kc, vc, pages, lens, prefix=prefix).out, *want, "prefixes")
    with pytest.raises(LoraError):
        step.paged_attention(torch.cat([q, q[:1]]), kc, vc, torch.cat([pages, pages[:1]]), torch.cat([lens, lens[:1]]))


def test_the_most_tokens():
    g, n, dim = gen(92), 1 << 20, 16
    kc, vc = small_cache(g, 9, 16, dim)
    q = torch.randn(n, 1, dim, generator=g, device="cuda").bfloat16()
    pages, lens, starts = ints([[3, 1, 8], [0, 2, 4]]), ints([37, 5]), ints([0, n // 2 + 3, n])
    for hint in (n, 1):
        r = step.paged_attention(q, kc, vc, pages, lens, starts=starts, max_rows=hint, causal=False)
        for b, (a, z) in enumerate(((0, n // 2 + 3), (n // 2 + 3, n))):
            k, v = (c[pages[b].long()].flatten(0, 1)[None, :lens[b].item(), 0] for c in (kc, vc))
            want = one_page(q[a:z], k, v, torch.ones(1, k.shape[1], dtype=torch.bool, device="cuda"))
            near(r.out[a:z], *want, f"request {b}")
    r = step.paged_attention(q, kc, vc, pages, lens, starts=starts, max_rows=n)
    assert (r.out[:n // 2 + 3 - 37] == 0).all() and (r.out[n // 2 + 3:n - 5] == 0).all() and (r.out[n - 1] != 0).any()
    kc, vc = (torch.zeros(n // 16, 16, 1, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    place = torch.randperm(n, generator=g, device="cuda").int()
    step.kv_append(q, -q, kc, vc, place)
    assert torch.equal(kc.flatten(0, 1)[place.long()], q) and torch.equal(vc.flatten(0, 1)[place.long()], -q)


def test_rows_past_32_bits():
    """Queries and results of more than 2^32 bytes and 2^31 elements."""
    g, n, heads, kv, dim = gen(93), (1 << 17) + 5, 160, 10, 128
    q = torch.randn(n, heads, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    kc, vc = (torch.randn(5, 16, kv, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    lens, starts = ints([70]), ints([0, n])
    r = step.paged_attention(q, kc, vc, ints([list(range(5))]), lens, starts=starts, max_rows=n, causal=False)
    for row in (0, n // 2, n - 200, n - 1):
        k, v = (c.flatten(0, 1)[:70].double().repeat_interleave(heads // kv, dim=1) for c in (kc, vc))
        x = q[row].double()
        p = torch.softmax((k * x).sum(dim=2) * dim ** -0.5, dim=0)[:, :, None]
        o = (p * v).sum(dim=0)
        # (p's and the result's rounding, and scores of 128 products of magnitudes below 30 in all: 130 x 30 x 2^-24)
        near(r.out[row], o, 2.0 ** -8 * o.abs() + (p * v.abs()).sum(dim=0) * (1.01 * 2.0 ** -8 + 2.0 ** -10), f"row {row}")
