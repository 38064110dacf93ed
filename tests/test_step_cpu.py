"""CPU-only checks of the serving-step operators' C ABI (include/step.h): the
built library exports exactly what the header declares, sizes workspaces, and
rejects bad arguments on the host before anything is launched (no GPU)."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

from tenant_lora_serving_amd import step

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, EUNSUP, EWS = 0, -1, -2, -3


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "step.h")).read(), flags=re.S)
    return sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(step.LIB_PATH):
        pytest.fail("libstep.so is not built (python -m tenant_lora_serving_amd.build)")
    return step.lib()


def test_library_exports_the_header(L):
    assert sorted(step.EXPORTED) == declared_functions()
    if not shutil.which("nm"):
        pytest.skip("nm is not available")
    out = subprocess.run(["nm", "-D", "--defined-only", step.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    syms = {ln.split()[-1] for ln in out.splitlines() if len(ln.split()) == 3 and ln.split()[1] == "T"}
    assert sorted(s for s in syms if not s.startswith("_Z")) == declared_functions()


def test_header_compiles_as_c():
    if not shutil.which("gcc"):
        pytest.skip("gcc is not available")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-x", "c",
                    os.path.join(ROOT, "include", "step.h")], check=True)


def test_status_strings(L):
    said = [L.step_status_string(s).decode() for s in (0, -1, -2, -3, -4)]
    assert said[0] == "ok" and len(set(said)) == 5
    assert L.step_status_string(7) == b"unknown status"


def test_norm_refusals(L):
    a = dict(x=0x1000, ldx=64, r=0x2000, ldr=64, w=0x3000, n=4, h=64, eps=1e-5, ro=0x4000, y=0x5000, q=0x6000,
             qs=0x7000)

    def call(**kw):
        v = dict(a, **kw)
        return L.step_rms_norm(v["x"], v["ldx"], v["r"], v["ldr"], v["w"], v["n"], v["h"], v["eps"], v["ro"],
                               v["y"], v["q"], v["qs"], None)
    assert call(n=0) == OK
    for bad in [dict(x=0), dict(x=0x1008), dict(ldx=56), dict(ldx=68), dict(r=0x2004), dict(ldr=60), dict(w=0),
                dict(w=0x3002), dict(n=-1), dict(h=0), dict(h=60), dict(eps=-1.0), dict(eps=math.nan),
                dict(eps=math.inf), dict(ro=0), dict(r=0), dict(ro=0x4008), dict(y=0x5004), dict(q=0x6004),
                dict(qs=0), dict(q=0), dict(y=0, q=0, qs=0), dict(r=0x2000, ro=0x2000, ldr=72)]:
        assert call(**bad) == EINVAL, bad
    assert call(h=32776, ldx=32776, ldr=32776) == EUNSUP
    assert call(n=(1 << 24) + 1) == EUNSUP


def linear(L, **kw):
    v = dict(x=0x1000, ldx=64, n=4, k=64, xq=0, ldxq=0, xs=0, w=0x2000, ws_=0, a=0x3000, b=0x4000, sc=0x5000, S=3,
             sizes=(24, 8), R=16, slot=0x6000, y=0x7000, ldy=32, ws=0x8000, bytes=1 << 20)
    v.update(kw)
    sizes = (ctypes.c_int32 * len(v["sizes"]))(*v["sizes"]) if v["sizes"] is not None else None
    return L.step_lora_linear(v["x"], v["ldx"], v["n"], v["k"], v["xq"], v["ldxq"], v["xs"], v["w"], v["ws_"], v["a"],
                              v["b"], v["sc"], v["S"], len(v["sizes"] or ()), sizes, v["R"], v["slot"], v["y"],
                              v["ldy"], v["ws"], v["bytes"], None)


def test_linear_refusals(L):
    assert linear(L, n=0) == OK
    assert linear(L, n=0, x=0, slot=0, y=0, ws=0) == OK
    for bad in [dict(x=0), dict(x=0x1002), dict(ldx=56), dict(ldx=68), dict(n=-1), dict(k=0), dict(k=24, ldx=24),
                dict(w=0), dict(w=0x2008), dict(a=0x3001), dict(b=0), dict(sc=0), dict(sc=0x5002), dict(S=0),
                dict(sizes=None), dict(sizes=()), dict(sizes=(8,) * 9), dict(sizes=(20, 8)), dict(sizes=(24, 0)),
                dict(slot=0), dict(slot=0x6001), dict(y=0), dict(y=0x7004), dict(ldy=24), dict(ldy=36),
                dict(xq=0x9000, ldxq=64, xs=0xa000), dict(xq=0x9000, ldxq=64, ws_=0xa000), dict(xs=0xa000),
                dict(ws_=0xa000), dict(xq=0x9000, ldxq=56, xs=0xa000, ws_=0xb000),
                dict(xq=0x9000, ldxq=72, xs=0xa000, ws_=0xb000), dict(xq=0x9008, ldxq=64, xs=0xa000, ws_=0xb000)]:
        assert linear(L, **bad) == EINVAL, bad
    for bad in [dict(R=12), dict(R=0), dict(R=136), dict(S=8193), dict(n=(1 << 18) + 1),
                dict(k=(1 << 18) + 16, ldx=(1 << 18) + 16), dict(sizes=((1 << 24) + 8,), ldy=1 << 25),
                dict(n=1 << 15, ldx=1 << 15), dict(n=1 << 15, xq=0x9000, ldxq=1 << 16, xs=0xa000, ws_=0xb000)]:
        assert linear(L, **bad) == EUNSUP, bad
    need = L.step_lora_linear_workspace_bytes(4, 64, 32, 2, 16)
    assert 0 < need < 1 << 20
    assert linear(L, bytes=need - 1) == EWS
    assert linear(L, ws=0, bytes=need) == EWS
    assert linear(L, ws=0x8008, bytes=need) == EWS


def test_linear_workspace_sizes(L):
    size = L.step_lora_linear_workspace_bytes
    assert size(4, 60, 32, 2, 16) == 0 and size(4, 64, 32, 9, 16) == 0 and size(4, 64, 32, 2, 12) == 0
    assert size(-1, 64, 32, 2, 16) == 0 and size((1 << 18) + 1, 64, 32, 2, 16) == 0
    # the inner sums of every row at least
    for n, k, out, l, r in [(1, 16, 8, 1, 8), (256, 4096, 6144, 3, 16), (6947, 4096, 28672, 2, 64),
                            (1 << 18, 16, 8, 8, 128)]:
        assert size(n, k, out, l, r) >= n * l * r * 4


def test_score_refusals(L):
    a = dict(z=0x1000, ld=100, f=0, n=2, v=100, t=0x2000, top=5, lp=0x3000, rk=0x4000, en=0x5000, ids=0x6000,
             tl=0x7000, ws=0x8000, bytes=1 << 20)

    def call(**kw):
        v = dict(a, **kw)
        return L.step_token_logprobs(v["z"], v["ld"], v["f"], v["n"], v["v"], v["t"], v["top"], v["lp"], v["rk"],
                                     v["en"], v["ids"], v["tl"], v["ws"], v["bytes"], None)
    assert call(n=0) == OK
    for bad in [dict(z=0), dict(z=0x1001), dict(z=0x1002, f=1), dict(ld=99), dict(n=-1), dict(v=0), dict(t=0),
                dict(t=0x2002), dict(top=-1), dict(lp=0), dict(rk=0x4001), dict(en=0), dict(ids=0), dict(tl=0),
                dict(top=0)]:
        assert call(**bad) == EINVAL, bad
    for bad in [dict(top=33), dict(n=(1 << 16) + 1), dict(v=(1 << 20) + 1, ld=1 << 21)]:
        assert call(**bad) == EUNSUP, bad
    need = L.step_token_logprobs_workspace_bytes(2, 100000, 5)
    assert need > 0
    assert call(v=100000, ld=100000, bytes=0) == EWS
    assert call(v=100000, ld=100000, ws=0, bytes=need) == EWS


def test_score_workspace_sizes(L):
    size = L.step_token_logprobs_workspace_bytes
    assert size(2, 0, 5) == 0 and size(2, 100, 33) == 0 and size(-1, 100, 0) == 0
    assert size(600, 1000, 0) == 0                  # a workgroup a row needs none
    for n, v, top in [(1, 128256, 5), (256, 128256, 20), (1 << 16, 1 << 20, 32), (512, 1 << 20, 0)]:
        parts = -(-(v // 8 + 2) // 4096)
        assert size(n, v, top) >= n * parts * (16 + 8 * top)


def test_binding_refuses_host_tensors():
    import torch
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        step.rms_norm(x, w)
    with pytest.raises(TypeError):
        step.token_logprobs(torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32), 1)
    with pytest.raises(TypeError):
        step.lora_linear(x, torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 8, 64), torch.zeros(1, 8, 8),
                         torch.ones(1), (8,), torch.zeros(2, dtype=torch.int32))
