"""What step.h's entry points accept, refuse and plan, on a host-only build of
them (step_abi.cpp and step_plan.cpp with the launchers replaced by the stubs
in step_host_stubs.cpp), so that accepted calls can be tested without a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tenant_lora_serving_amd", "csrc")
OK, EINVAL, EUNSUP, EWS = 0, -1, -2, -3
NORM, LINEAR, SCORE = range(3)


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ is not available")
    path = str(tmp_path_factory.mktemp("step") / "libstep_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
                    "-I", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    os.path.join(CSRC, "step_abi.cpp"), os.path.join(CSRC, "step_plan.cpp"),
                    os.path.join(ROOT, "tests", "step_host_stubs.cpp"), "-o", path], check=True)
    L = ctypes.CDLL(path)
    i32, i64, p, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    L.step_lora_linear.argtypes = [p, i64, i32, i32, p, i64, p, p, p, p, p, p, i32, i32, p, i32, p, p, i64, p, sz, p]
    L.step_token_logprobs.argtypes = [p, i64, i32, i32, i32, p, i32, p, p, p, p, p, p, sz, p]
    L.step_lora_linear_workspace_bytes.restype = L.step_token_logprobs_workspace_bytes.restype = sz
    L.step_lora_linear_workspace_bytes.argtypes = [i32] * 5
    L.step_token_logprobs_workspace_bytes.argtypes = [i32] * 3
    L.stub_calls.restype = ctypes.c_longlong
    return L


@pytest.fixture(autouse=True)
def reset(L):
    L.stub_reset()


def score(L, n, v, top, ws_bytes, fp32=0):
    tops = (0x6000, 0x7000) if top else (None, None)
    return L.step_token_logprobs(0x1000, v, fp32, n, v, 0x2000, top, 0x3000, 0x4000, 0x5000, *tops, 0x8000, ws_bytes,
                                 None)


VOCABS = [1, 4096, 4097, 8180, 8190, 32000, 32750, 32760, 32770, 65500, 128256, 262143, 262144, 524288, 1 << 20]


@pytest.mark.parametrize("v", VOCABS)
def test_score_workspace_serves_every_smaller_batch(L, v):
    """A workspace sized for n rows is accepted for any fewer rows, whatever the type."""
    size, top = L.step_token_logprobs_workspace_bytes, 5
    rows = [*range(1, 140), 170, 171, 255, 256, 257, 300, 511, 512, 513, 700, 1 << 16]
    sizes = [size(n, v, top) for n in rows]
    assert sizes == sorted(sizes)
    for most, have in zip(rows, sizes):
        for n in rows:
            if n > most:
                break
            for fp32 in (0, 1):
                assert score(L, n, v, top, have, fp32) == OK, (most, n, fp32)


def test_score_workspace_grows_with_every_size(L):
    size = L.step_token_logprobs_workspace_bytes
    for n in (1, 100, 512, 3000):
        for top in (0, 5, 32):
            by_v = [size(n, v, top) for v in VOCABS]
            assert by_v == sorted(by_v)
        for v in VOCABS:
            by_top = [size(n, v, top) for top in range(33)]
            assert by_top == sorted(by_top)


def test_linear_workspace_grows_with_every_size(L):
    size = L.step_lora_linear_workspace_bytes
    for out in (8, 96, 6144, 8192, 32008, 1 << 20):
        by_n = [size(n, 4096, out, 3, 16) for n in range(1, 400)]
        assert by_n == sorted(by_n)
    for n in (1, 64, 65, 128, 256, 257):
        by_out = [size(n, 4096, out, 3, 16) for out in range(8, 40000, 8)]
        assert by_out == sorted(by_out)


def test_shapes_are_computed_in_the_tiles_that_they_test(L):
    import test_gpu_step_tiles as T
    listed = T.ALL + [(256256, (fp8, *case)) for fp8 in (False, True) for case in (T.BROKEN[fp8], T.SLOTS)]
    for tile, (fp8, n, k, widths, S, R) in listed:
        assert L.stub_linear_tile(n, k, sum(widths), len(widths), R, int(fp8)) == tile, (tile, fp8, n, k, widths)
    assert len({tile for tile, _ in listed}) == 10     # every kind
    assert {tile for tile, case in T.ALL if case[0]} == {tile for tile, case in T.ALL if not case[0]}


def linear(L, **kw):
    v = dict(x=0x1000, ldx=64, n=4, k=64, xq=None, ldxq=0, xs=None, w=0x2000, ws_=None, a=0x3000, b=0x4000, sc=0x5000,
             S=3, sizes=(24, 8), R=16, slot=0x6000, y=0x7000, ldy=32, ws=0x8000, bytes=1 << 40)
    v.update(kw)
    sizes = (ctypes.c_int32 * len(v["sizes"]))(*v["sizes"])
    return L.step_lora_linear(v["x"], v["ldx"], v["n"], v["k"], v["xq"], v["ldxq"], v["xs"], v["w"], v["ws_"], v["a"],
                              v["b"], v["sc"], v["S"], len(sizes), sizes, v["R"], v["slot"], v["y"], v["ldy"],
                              v["ws"], v["bytes"], None)


FP8 = dict(xq=0x9000, xs=0xa000, ws_=0xb000)


def test_linear_spans(L):
    """Row offsets are 32-bit in the kernels: strides that pass them are refused,
    also ones whose product with n wraps around 64 bits."""
    for n in (1, 3, 1 << 18):
        most = ((1 << 30) - 1) // n // 8 * 8
        assert linear(L, n=n, ldx=most) == OK
        most8 = ((1 << 31) - 1) // n // 16 * 16
        assert linear(L, n=n, ldxq=most8, **FP8) == OK
        assert L.stub_calls(LINEAR) == 2
        for ld in (most + 8, 1 << 30, 1 << 45, 1 << 46, 1 << 47, 3 << 46, 1 << 61, (1 << 63) - 8):
            assert linear(L, n=n, ldx=ld) == EUNSUP, (n, ld)
        for ld in (most8 + 16, 1 << 31, 1 << 46, 1 << 47, 3 << 46, 1 << 61, (1 << 63) - 16):
            assert linear(L, n=n, ldxq=ld, **FP8) == EUNSUP, (n, ld)
        assert L.stub_calls(LINEAR) == 2
        L.stub_reset()
    assert linear(L, n=0, ldx=1 << 40) == OK and L.stub_calls(LINEAR) == 0


def test_linear_grid_of_small_tiles(L):
    """8-bit rows of short k run in 64-row tiles only: past 10^11 results their
    grid would pass 2^32 threads."""
    n = 1 << 18
    for out, want in (((10 ** 11 - 1) // n // 8 * 8, OK), (10 ** 11 // n // 8 * 8 + 8, EUNSUP), (1 << 24, EUNSUP)):
        assert linear(L, n=n, k=16, ldxq=16, sizes=(out,), ldy=out, **FP8) == want
        assert linear(L, n=n, k=272, ldx=272, ldxq=272, sizes=(out,), ldy=out, **FP8) == OK
        assert linear(L, n=n, k=16, sizes=(out,), ldy=out) == OK
        tile = L.stub_linear_tile(n, 16, out, 1, 16, 1)
        if want == OK:
            rows, cols = tile // 1000, tile % 1000
            assert -(-n // rows) * (-(-out // cols) + 7) * 256 < 1 << 32


def test_binding_refuses_sizes_past_32_bits():
    """The library takes 32-bit sizes; a larger one must not arrive there as its low half."""
    from tenant_lora_serving_amd import step
    from tenant_lora_serving_amd.lora import LoraError
    if not os.path.exists(step.LIB_PATH):
        pytest.fail("libstep.so is not built (python -m tenant_lora_serving_amd.build)")
    far = 1 << 32
    for sizes in ((far + 2, 100, 5), (2, far + 100, 5), (2, 100, far + 5)):
        with pytest.raises(LoraError) as e:
            step.logprobs_workspace(*sizes, device="cpu")
        assert e.value.status == EUNSUP
    for sizes in ((far + 4, 64, 32, 2, 16), (4, far + 64, 32, 2, 16), (4, 64, far + 32, 2, 16), (4, 64, 32, far + 2, 16),
                  (4, 64, 32, 2, far + 16)):
        with pytest.raises(LoraError) as e:
            step.linear_workspace(*sizes, device="cpu")
        assert e.value.status == EUNSUP
