"""Appending to the paged cache against its 64-bit definition, bit by bit where nothing is computed.

A turned value is two products and a sum in fp32, off by at most 2^-22 (|a cos| + |b sin|), and is rounded once:
2^-8 of it in bf16, 2^-4 in e4m3 (or half of e4m3's smallest step, 2^-10)."""
import math

import pytest
import torch

from tenant_lora_serving_amd import step
from tenant_lora_serving_amd.lora import LoraError

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pool(g, pages, page, kv, dim, cache, layout):
    shape = {"apart": (2, pages, page, kv, dim), "heads": (2, pages, kv, page, dim), "joint": (pages, 2, page, kv, dim)}[layout]
    t = torch.randn(shape, generator=g, device="cuda").to(torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16)
    if layout == "joint":
        return t[:, 0], t[:, 1]
    return (t[0], t[1]) if layout == "apart" else (t[0].transpose(1, 2), t[1].transpose(1, 2))


def turned(x, positions, rotation, neighbours):
    """(values, magnitudes) in 64 bits."""
    x = x.double()
    mag = x.abs()
    if rotation is None:
        return x, mag
    rot = rotation.shape[1]
    row = rotation.double()[positions.long()][:, None, :]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, rot // 2), slice(rot // 2, rot))
    y, m = x.clone(), mag.clone()
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    m[..., a] = (x[..., a] * cos).abs() + (x[..., b] * sin).abs()
    m[..., b] = (x[..., b] * cos).abs() + (x[..., a] * sin).abs()
    return y, m


def close(got, want, mag, step_rel, step_abs, what):
    err, tol = (got.double() - want).abs(), want.abs() * step_rel + step_abs + mag * 2.0 ** -22 * (1 + step_rel)
    assert (err <= tol).all(), f"{what}: {(err > tol).sum()} of {err.numel()} off"


def check(n, heads=4, kv=2, dim=64, rot=64, cache="bf16", layout="apart", neighbours=False, page=16, q=True, pad=0, seed=1,
          in_place=False, place=None):
    g = gen(seed)
    qkv = torch.randn(n, (heads + 2 * kv) * dim + pad, generator=g, device="cuda").bfloat16()
    parts = [p.unflatten(1, (-1, dim)) for p in qkv[:, :(heads + 2 * kv) * dim].split([heads * dim, kv * dim, kv * dim], dim=1)]
    pages = n // page + 5
    kc, vc = pool(g, pages, page, kv, dim, cache, layout)
    before = [c.double() for c in (kc, vc)]
    if place is None:
        place = torch.randperm(pages * page, generator=g, device="cuda")[:n].int()
        place[torch.rand(n, generator=g, device="cuda") < 0.1] = -1
    table = step.rotation_table(500, rot, 1e4) if rot else None
    positions = torch.randint(0, 500, (n,), generator=g, device="cuda").int() if rot else None
    scales = dict(k_scale=0.005 * (1 + torch.rand(kv, generator=g, device="cuda")),
                  v_scale=0.005 * (1 + torch.rand(kv, generator=g, device="cuda"))) if cache == "e4m3" else {}
    want_q, mag_q = turned(parts[0], positions, table, neighbours)
    want_k, mag_k = turned(parts[1], positions, table, neighbours)
    got = step.kv_append(parts[1], parts[2], kc, vc, place, q=parts[0] if q else None, positions=positions, rotation=table,
                         neighbours=neighbours, q_out=parts[0] if in_place else None, **scales)
    what = f"{n} {heads}/{kv} {dim} {rot} {cache} {layout}"
    if q:
        close(got, want_q, mag_q, 2.0 ** -8, 0.0, what + " q")
        if not rot:
            assert torch.equal(got.double(), want_q)
    else:
        assert got is None
    live = (place >= 0) & (place < pages * page)
    at = place[live].long()
    for c, old, values, mag, scale in ((kc, before[0], want_k, mag_k, scales.get("k_scale")),
                                       (vc, before[1], parts[2].double(), parts[2].double().abs(), scales.get("v_scale"))):
        new = c.double()
        if scale is not None:
            values, mag = values / scale.double()[:, None], mag / scale.double()[:, None]
            values = values.clamp(-448, 448)
            close(new[at // page, at % page], values[live], mag[live], 2.0 ** -4, 2.0 ** -10, what)
        else:
            close(new[at // page, at % page], values[live], mag[live], 2.0 ** -8, 0.0, what)
        if scale is None and (c is vc or not rot):
            assert torch.equal(new[at // page, at % page], values[live])
        new[at // page, at % page] = old[at // page, at % page]
        assert torch.equal(new, old), what + ": another place of the cache changed"


@pytest.mark.parametrize("n", [1, 2, 37, 500, 3000, 5001])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_sizes(n, cache, neighbours):
    check(n, cache=cache, neighbours=neighbours)


@pytest.mark.parametrize("dim,rot", [(16, 16), (16, 0), (64, 16), (80, 32), (96, 96), (128, 128), (128, 48), (208, 0), (256, 256)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("neighbours", [False, True])
def test_columns(dim, rot, cache, neighbours):
    check(19, dim=dim, rot=rot, cache=cache, neighbours=neighbours, heads=6, kv=3, pad=24)


@pytest.mark.parametrize("layout", ["apart", "joint", "heads"])
@pytest.mark.parametrize("page", [1, 7, 128])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_layouts(layout, page, cache):
    check(300, layout=layout, page=page, cache=cache, pad=8)
    check(5, heads=64, kv=1, layout=layout, page=page, cache=cache)


def test_without_queries_and_in_place():
    check(33, q=False)
    check(33, q=False, rot=0)
    check(33, in_place=True)
    check(4100, in_place=True, neighbours=True, rot=32)


def test_places_outside_the_cache():
    place = torch.tensor([-1, -2 ** 31, 2 ** 31 - 1, 5 * 16, 5 * 16 - 1, 3], dtype=torch.int32, device="cuda")
    check(6, place=place)
    check(6, place=place, cache="e4m3")


def test_positions_outside_the_rotation():
    g = gen(3)
    x = torch.randn(4, 2, 32, generator=g, device="cuda").bfloat16()
    kc, vc = pool(g, 2, 4, 2, 32, "bf16", "apart")
    before = kc.clone(), vc.clone()
    positions = torch.tensor([-1, 10, 9, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    place = torch.arange(4, dtype=torch.int32, device="cuda")
    q = step.kv_append(x, x, kc, vc, place, q=x, positions=positions, rotation=step.rotation_table(10, 16))
    assert torch.isnan(q[[0, 1, 3]]).all() and torch.isfinite(q[2]).all()
    for c, old in zip((kc, vc), before):
        assert torch.equal(c[0, [0, 1, 3]], old[0, [0, 1, 3]]) and torch.equal(c[1], old[1])
    assert torch.equal(vc[0, 2], x[2])


def test_values_out_of_range_and_not_finite():
    x = torch.zeros(1, 1, 16, device="cuda", dtype=torch.bfloat16)
    x[0, 0, :8] = torch.tensor([1e30, -1e30, math.inf, -math.inf, math.nan, 448.0, 465.0, -1e-30], device="cuda")
    kc, vc = (torch.zeros(1, 1, 1, 16, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    one = torch.ones(1, device="cuda")
    step.kv_append(x, x, kc, vc, torch.zeros(1, dtype=torch.int32, device="cuda"), k_scale=one, v_scale=one)
    for c in (kc, vc):
        got = c.float()[0, 0, 0]
        assert got[:4].tolist() == [448.0, -448.0, 448.0, -448.0] and math.isnan(got[4].item())
        assert got[5:8].tolist() == [448.0, 448.0, 0.0]
    kc, vc = (torch.zeros(1, 1, 1, 16, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    step.kv_append(x, x, kc, vc, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(kc.view(torch.int16), x.view(torch.int16).reshape(kc.shape))


def test_two_tokens_with_one_place():
    """Every 16 bytes of the place are one of the two tokens'."""
    k = torch.stack([torch.full((2, 64), float(i + 1)) for i in range(2)]).cuda().bfloat16()
    kc, vc = (torch.zeros(2, 4, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    step.kv_append(k, k, kc, vc, torch.tensor([5, 5], dtype=torch.int32, device="cuda"))
    for c in (kc, vc):
        parts = c[1, 1].reshape(-1, 8)
        assert ((parts == 1).all(dim=1) | (parts == 2).all(dim=1)).all()
        c[1, 1] = 0
        assert (c == 0).all()


def test_a_cache_past_32_bits():
    far = torch.zeros(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    kc, vc = (far.as_strided((3, 4, 2, 64), (2 ** 30, 128, 64, 1), at) for at in (0, 4096))
    x = torch.randn(2, 2, 64, generator=gen(4), device="cuda").bfloat16()
    step.kv_append(x, -x, kc, vc, torch.tensor([11, 6], dtype=torch.int32, device="cuda"))
    for c, y in ((kc, x), (vc, -x)):
        assert torch.equal(c[2, 3], y[0]) and torch.equal(c[1, 2], y[1])


def test_the_table():
    t = step.rotation_table(131072, 64, 5e5)
    assert t.shape == (131072, 64) and t.dtype == torch.float32
    at = 131071 * 5e5 ** (-2 * 3 / 64)
    assert abs(t[-1, 3].item() - math.cos(at)) < 1e-7 and abs(t[-1, 35].item() - math.sin(at)) < 1e-7
    with pytest.raises(ValueError):
        step.rotation_table(10, 7)


def test_graph():
    g = gen(9)
    k, v, q = (torch.randn(9, h, 64, generator=g, device="cuda").bfloat16() for h in (2, 2, 8))
    kc, vc = (torch.zeros(8, 16, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    place, pos = (torch.arange(9, dtype=torch.int32, device="cuda") for _ in range(2))
    table = step.rotation_table(100, 64)
    call = lambda: step.kv_append(k, v, kc, vc, place, q=q, positions=pos, rotation=table)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for i in range(3):
        place.copy_(torch.randperm(128, device="cuda")[:9])
        pos.copy_(torch.randint(0, 100, (9,), device="cuda"))
        q.normal_(generator=g), k.normal_(generator=g)
        kc.zero_(), vc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = held.clone(), kc.clone(), vc.clone()
        kc.zero_(), vc.zero_()
        again = call()
        assert all(torch.equal(x, y) for x, y in zip(got, (again, kc, vc)))
        s = torch.cuda.Stream()
        other = step.kv_append(k, v, kc, vc, place, q=q, positions=pos, rotation=table, stream=s)
        s.synchronize()
        assert torch.equal(other, again)


def test_refusals():
    g = gen(5)
    k, v = (torch.randn(3, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    kc, vc = pool(g, 4, 8, 2, 64, "bf16", "apart")
    place = torch.zeros(3, dtype=torch.int32, device="cuda")
    pos, table, one = place.clone(), step.rotation_table(10, 64), torch.ones(2, device="cuda")
    ok = dict(k=k, v=v, k_cache=kc, v_cache=vc, place=place)

    def call(**kw):
        a = dict(ok, **kw)
        return step.kv_append(a.pop("k"), a.pop("v"), a.pop("k_cache"), a.pop("v_cache"), a.pop("place"), **a)
    for bad in (dict(k=k.cpu()), dict(k=k.float()), dict(v=v.half()), dict(place=place.long()), dict(k_cache=kc.float()),
                dict(k_cache=kc.to(torch.float8_e4m3fn), k_scale=one, v_scale=one), dict(rotation=table.double(), positions=pos)):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(v=v[:2]), dict(k=k[:, :, ::2]), dict(place=place[:2]), dict(k_cache=kc[:, :, :1]), dict(v_cache=vc[:2]),
                dict(k_cache=kc.transpose(1, 2)), dict(k_scale=one, v_scale=one), dict(positions=pos), dict(rotation=table),
                dict(q_out=k), dict(q=k, q_out=k[:2]), dict(rotation=table, positions=pos[:2]),
                dict(k_cache=kc.to(torch.float8_e4m3fn), v_cache=vc.to(torch.float8_e4m3fn))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(rotation=step.rotation_table(10, 24), positions=pos), dict(rotation=step.rotation_table(10, 80), positions=pos),
                dict(q=k[:, :1], q_out=None)):
        with pytest.raises((LoraError, ValueError)):
            call(**bad)
    assert call(k=k[:0], v=v[:0], place=place[:0], q=k[:0]).shape == (0, 2, 64)
