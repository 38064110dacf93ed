"""The paged cache's entry points (include/step.h) on a host-only build of them: what they accept
and refuse, which kernels a call takes, and how an attention call is divided among workgroups."""
import ctypes
import math
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tenant_lora_serving_amd", "csrc")
OK, EINVAL, EUNSUP, EWS = 0, -1, -2, -3
FEW, MANY, APPEND = range(3)


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ is not available")
    path = str(tmp_path_factory.mktemp("attend") / "libattend_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, "attend_abi.cpp"),
                    os.path.join(ROOT, "tests", "attend_host_stubs.cpp"), "-o", path], check=True)
    L = ctypes.CDLL(path)
    from tenant_lora_serving_amd import step
    real = step.lib()
    for name in ("step_kv_append", "step_paged_attention", "step_paged_attention_workspace_bytes"):
        getattr(L, name).argtypes = getattr(real, name).argtypes
        getattr(L, name).restype = getattr(real, name).restype
    return L


@pytest.fixture(autouse=True)
def reset(L):
    L.stub_reset()


def launches(L):
    got = []
    for i in range(L.stub_count()):
        v = (ctypes.c_int * 5)()
        L.stub_launch(i, v)
        got.append(list(v))
    return got


# ---------------------------------------------------------------- refusals
APPENDED = dict(q=0x10000, ldq=512, k=0x20000, ldk=256, v=0x30000, ldv=256, n=5, heads=4, kv=2, dim=128, pos=0x40000,
                rotation=0x50000, rows=100, rot=128, neighbours=0, place=0x60000, kc=0x70000, vc=0x80000, ps=4096, ts=256,
                hs=128, pages=3, page=16, ks=0, vs=0, qo=0x90000, ldo=512)


def append(L, **kw):
    a = dict(APPENDED, **kw)
    return L.step_kv_append(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["n"], a["heads"], a["kv"], a["dim"],
                            a["pos"], a["rotation"], a["rows"], a["rot"], a["neighbours"], a["place"], a["kc"], a["vc"],
                            a["ps"], a["ts"], a["hs"], a["pages"], a["page"], a["ks"], a["vs"], a["qo"], a["ldo"], None)


CACHE_REFUSED = [dict(kc=0), dict(vc=0x80008), dict(ps=4100), dict(ts=120), dict(hs=64), dict(hs=132), dict(pages=0),
                 dict(page=0), dict(ks=0x100), dict(vs=0x100), dict(ks=0x102, vs=0x200), dict(ks=0x100, vs=0x200, hs=136),
                 dict(kv=0), dict(kv=3), dict(dim=0), dict(dim=120), dict(n=-1)]
CACHE_UNSUPPORTED = [dict(pages=1 << 20, page=1 << 12), dict(ps=1 << 35), dict(n=(1 << 20) + 1),
                     dict(dim=272, ldq=4096, ldk=4096, ldv=4096, ldo=4096, hs=272, ts=1088, ps=1 << 20)]


def test_append_refusals(L):
    assert append(L) == OK and launches(L) == [[APPEND, 0, 0, 0, 0]]
    for good in [dict(q=0, qo=0, heads=0), dict(rot=0, pos=0, rotation=0), dict(ks=0x100, vs=0x200), dict(rot=16),
                 dict(pages=1, ps=3), dict(page=1, ts=-5), dict(kv=1, hs=1), dict(qo=0x10000), dict(neighbours=1)]:
        assert append(L, **good) == OK, good
    L.stub_reset()
    assert append(L, n=0, q=0, qo=0, k=0, v=0, place=0) == OK
    for bad in CACHE_REFUSED + [
            dict(q=0), dict(qo=0), dict(q=0x10008), dict(ldq=504), dict(ldq=516), dict(k=0), dict(ldk=248), dict(v=8),
            dict(ldv=252), dict(pos=0), dict(rotation=0), dict(rotation=0x50004), dict(rows=0), dict(rot=-16), dict(rot=24),
            dict(rot=144), dict(place=0), dict(place=2), dict(qo=0x10000, ldo=520), dict(ldo=500)]:
        assert append(L, **bad) == EINVAL, bad
    for bad in CACHE_UNSUPPORTED + [dict(ldq=1 << 40), dict(ldk=1 << 40), dict(heads=4098, kv=2),
                                    dict(heads=130, kv=2, ldq=1 << 15, ldo=1 << 15)]:
        assert append(L, **bad) == EUNSUP, bad
    assert launches(L) == []


ATTENDED = dict(q=0x10000, ldq=512, n=5, requests=5, heads=4, kv=2, dim=128, kc=0x70000, vc=0x80000, ps=4096, ts=256,
                hs=128, pages=3, page=16, ks=0, vs=0, table=0x1000, ldt=8, cols=8, lens=0x2000, starts=0, max_rows=1,
                causal=1, scale=0.1, prefixes=0, pt=0, ldp=0, pcols=0, pl=0, pst=0, out=0x90000, ldo=512, lse=0,
                ws=0xa0000, bytes=1 << 40)
PREFIXED = dict(prefixes=2, pt=0x3000, ldp=6, pcols=6, pl=0x4000, pst=0x5000)


def attend(L, **kw):
    a = dict(ATTENDED, **kw)
    return L.step_paged_attention(a["q"], a["ldq"], a["n"], a["requests"], a["heads"], a["kv"], a["dim"], a["kc"],
                                  a["vc"], a["ps"], a["ts"], a["hs"], a["pages"], a["page"], a["ks"], a["vs"],
                                  a["table"], a["ldt"], a["cols"], a["lens"], a["starts"], a["max_rows"], a["causal"],
                                  a["scale"], a["prefixes"], a["pt"], a["ldp"], a["pcols"], a["pl"], a["pst"], a["out"],
                                  a["ldo"], a["lse"], a["ws"], a["bytes"], None)


def test_attention_refusals(L):
    for good in [{}, PREFIXED, dict(starts=0x6000, requests=2, max_rows=4), dict(lse=0x7000), dict(cols=0, ldt=0, table=0),
                 dict(PREFIXED, pcols=0, ldp=0, pt=0), dict(ks=0x100, vs=0x200), dict(ldq=1024, ldo=1024),
                 dict(pages=1, ps=7, page=1, ts=3, kv=1, heads=4, hs=2)]:
        assert attend(L, **good) == OK, good
    L.stub_reset()
    assert attend(L, n=0, requests=0, q=0, out=0, lens=0, table=0, ws=0) == OK
    assert attend(L, n=5, requests=0, starts=0x6000) == OK
    for bad in CACHE_REFUSED + [
            dict(q=0), dict(q=0x10008), dict(ldq=504), dict(ldq=516), dict(requests=4), dict(requests=-1, starts=0x6000),
            dict(starts=0x6000, max_rows=0), dict(starts=0x6002), dict(table=0), dict(table=2), dict(ldt=7), dict(cols=-1),
            dict(lens=0), dict(lens=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e-31),
            dict(scale=1e31),
            dict(out=0), dict(out=0x90008), dict(ldo=504), dict(ldo=516), dict(lse=2), dict(prefixes=-1),
            dict(PREFIXED, pt=0), dict(PREFIXED, ldp=5), dict(PREFIXED, pl=0), dict(PREFIXED, pst=0),
            dict(PREFIXED, pcols=-1)]:
        assert attend(L, **bad) == EINVAL, bad
    for bad in CACHE_UNSUPPORTED + [
            dict(cols=1 << 21, ldt=1 << 21), dict(PREFIXED, pcols=1 << 21, ldp=1 << 21), dict(ldt=1 << 40),
            dict(requests=(1 << 16) + 1, starts=0x6000), dict(PREFIXED, prefixes=(1 << 16) + 1),
            dict(heads=130, kv=2, ldq=1 << 15, ldo=1 << 15), dict(ldq=1 << 40), dict(ldo=1 << 40)]:
        assert attend(L, **bad) == EUNSUP, bad
    need = L.step_paged_attention_workspace_bytes(5, 4, 2, 128, 0)
    assert attend(L, bytes=need - 1) == EWS and attend(L, ws=0) == EWS and attend(L, ws=0xa0008) == EWS
    assert attend(L, bytes=need, **PREFIXED) == EWS
    assert launches(L) == []
    assert attend(L, bytes=need) == OK
    assert attend(L, bytes=L.step_paged_attention_workspace_bytes(5, 4, 2, 128, 1), **PREFIXED) == OK


def test_workspace_sizes(L):
    size = L.step_paged_attention_workspace_bytes
    assert size(-1, 4, 2, 128, 0) == 0 and size(5, 4, 3, 128, 0) == 0 and size(5, 4, 2, 120, 0) == 0
    assert size(5, 4, 2, 128, -1) == 0 and size((1 << 20) + 1, 4, 2, 128, 0) == 0
    for dim in (16, 64, 80, 128, 256):
        for heads, kv in ((4, 2), (64, 1), (4096, 4096)):
            plain = [size(n, heads, kv, dim, 0) for n in (0, 1, 7, 256, 5000, 1 << 20)]
            both = [size(n, heads, kv, dim, 3) for n in (0, 1, 7, 256, 5000, 1 << 20)]
            assert len(set(plain)) == 1 and both == sorted(both) and both[0] >= plain[0]
            # what every row brings from its prefix: sums of values, a maximum and a sum
            assert both[-1] - plain[-1] >= (1 << 20) * heads * (dim + 2) * 4


def test_which_kernels(L):
    attend(L)
    attend(L, heads=34, kv=2, ldq=1 << 13, ldo=1 << 13)              # 17 heads to a key head
    attend(L, starts=0x6000, requests=2, max_rows=4, n=8)            # 8 rows of a tile
    attend(L, starts=0x6000, requests=2, max_rows=9, n=18)
    attend(L, **PREFIXED)
    assert [x[0] for x in launches(L)] == [FEW, MANY, FEW, MANY, FEW, FEW]
    assert launches(L)[4][2:] == [4, 0, 1] and launches(L)[5][2:] == [5, 1, 0]
    L.stub_reset()
    attend(L, n=256, requests=256, **PREFIXED)                       # 128 requests a prefix
    assert [x[0] for x in launches(L)] == [MANY, FEW]
    # no more workgroups than work that the tables allow: 5 requests of 2 heads, at most 128 keys
    assert launches(L)[1][1] <= 512
    L.stub_reset()
    attend(L, n=1, requests=1)
    assert 1 <= launches(L)[0][1] <= 8


def test_binding_refuses_host_tensors():
    import torch
    from tenant_lora_serving_amd import step
    x, cache = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 4, 64, dtype=torch.bfloat16)
    at = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        step.kv_append(x, x, cache, cache, at)
    with pytest.raises(TypeError):
        step.paged_attention(x, cache, cache, torch.zeros(2, 1, dtype=torch.int32), at)
    with pytest.raises(ValueError):
        step.rotation_table(10, 0, device="cpu")
    t = step.rotation_table(4, 2, device="cpu")
    assert t.dtype == torch.float32 and t.tolist() == [[pytest.approx(math.cos(i)), pytest.approx(math.sin(i))] for i in range(4)]


# ---------------------------------------------------------------- pages
def test_page_of(L):
    for page in [1, 2, 3, 5, 7, 8, 16, 24, 100, 127, 128, 129, 1000, 4095, 65536, 65537, 1 << 23, (1 << 24) - 1, 1 << 24]:
        keys = {0, 1, 2, (1 << 24) - 1, (1 << 24) - 2}
        for m in {1, 2, 3, (1 << 24) // page, (1 << 24) // page - 1, (1 << 23) // page}:
            keys |= {m * page - 1, m * page, m * page + 1}
        for key in keys:
            if 0 <= key < 1 << 24:
                assert L.stub_page_of(page, key) == key // page, (page, key)


# ---------------------------------------------------------------- division
def divide(L, rows, lens, kv, tokens, causal, groups, least, whole, step, fixed):
    arr = ctypes.c_int * len(rows)
    most = 200000
    to = (ctypes.c_int * (12 * most))()
    n = L.stub_divide(len(rows), arr(*rows), arr(*lens), kv, tokens, causal, groups, fixed, least, whole, step, to,
                      most)
    assert n >= 0
    return [tuple(to[12 * k:12 * k + 12]) for k in range(n)]


def check_division(L, rows, lens, kv, tokens, causal, groups, least, whole, step, fixed=64):
    pieces = divide(L, rows, lens, kv, tokens, causal, groups, least, whole, step, fixed)
    by_tile, slots, tickets = {}, set(), {}
    for w, j, g, i, keys, lo, hi, begins, split, first, count, slot in pieces:
        by_tile.setdefault((j, g, i), []).append((w, keys, lo, hi, begins, split, first, count, slot))
    want = {(j, g, i) for j, r in enumerate(rows) for g in range(kv) for i in range(-(-r // tokens))}
    assert set(by_tile) == want
    per_group = {}
    for (j, g, i), parts in by_tile.items():
        last = i == -(-rows[j] // tokens) - 1
        see = lens[j] if not causal or last else max(0, lens[j] - rows[j] + (i + 1) * tokens)
        at = 0
        assert [p[0] for p in parts] == list(range(parts[0][0], parts[0][0] + len(parts)))
        for w, keys, lo, hi, begins, split, first, count, slot in parts:
            assert keys == see and lo == at and lo <= hi and (hi == keys or hi % step == 0)
            at = hi
            assert bool(begins) == (w == parts[0][0]) and bool(split) == (len(parts) > 1)
            per_group[w] = per_group.get(w, 0) + hi - lo + fixed
            if split:
                assert first == parts[0][0] and count == len(parts)
                assert slot >= 0 and slot // 2 == w and slot not in slots
                slots.add(slot)
                assert tickets.setdefault(first, (j, g, i)) == (j, g, i)
        assert at == see
    return per_group


@pytest.mark.parametrize("seed", range(60))
def test_division_covers_every_key_once(L, seed):
    rng = random.Random(seed)
    jobs = rng.choice([1, 1, 2, 5, 40, 300])
    causal = rng.random() < 0.6
    top_rows = rng.choice([1, 1, 3, 200, 2000]) if jobs < 100 else rng.choice([1, 20])
    rows = [rng.choice([0, 1, rng.randint(0, top_rows)]) for _ in range(jobs)]
    top = rng.choice([1, 10, 100, 1000, 20000])
    lens = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(jobs)]
    kv, tokens = rng.choice([1, 2, 8]), rng.choice([1, 4, 5, 16, 32, 128])
    few = rng.random() < 0.5
    groups = rng.choice([1, 2, 7, 64, 512])
    check_division(L, rows, lens, kv, tokens, causal, groups, 128, 256 if few else 1024, 128 if few else 64,
                   rng.choice([64, 256]))


def test_division_is_even(L):
    """One long request among short ones does not hold up the rest."""
    rng = random.Random(1)
    lens = [rng.randint(50, 500) for _ in range(200)] + [30000]
    load = check_division(L, [1] * 201, lens, 8, 4, 1, 512, 128, 256, 128)
    total = 8 * sum(x + 64 for x in lens)
    assert max(load.values()) <= 1.3 * total / 512 + 256 + 128


def test_division_of_the_largest_sums(L):
    """2^20 rows that see 2^24 keys each: costs pass 32 bits."""
    n, keys = 1 << 20, 1 << 24
    check_division(L, [n], [keys], 1, 2048, 1, 512, 128, 1024, 64)
    check_division(L, [n // 2, 0, n // 2], [keys, keys, 100], 1, 1024, 1, 512, 128, 1024, 64)
