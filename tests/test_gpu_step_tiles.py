"""step_lora_linear in every kind of tile, against its definition in 64 bits on
the GPU (tolerances as in test_gpu_step.py).  test_step_host_cpu.py asserts that
the shapes listed here are computed in the tiles that they are listed under."""
import math

import pytest
import torch

from tenant_lora_serving_amd import step
from test_gpu_step import check_linear, gen, linear64, linear_inputs, randn, within

pytestmark = pytest.mark.gpu

# (fp8, n, k, widths, S, R).  256 x 256 tiles: rows and columns that do not fill
# the last tile and that do, columns of tiles that are and are not a multiple of
# four, slices that end inside a tile, k shorter than a line, with a ragged last
# line and of whole lines, every count of lines of an adapter, tiles that name
# one slot, a few and hundreds.
LARGE = [
    (False, 2100, 16, (3992,), 5, 8),
    (False, 2100, 272, (3992,), 5, 8),
    (False, 2304, 512, (3840,), 3, 16),
    (False, 2049, 1040, (1000, 2000, 1096), 30, 24),
    (False, 4097, 320, (2056,), 1, 128),
    (False, 2100, 640, (2048, 2040), 700, 8),
    (False, 16000, 144, (520,), 64, 64),
    (False, 2300, 192, (136, 8, 3800), 2300, 32),
    (True, 2100, 272, (3992,), 5, 8),
    (True, 2304, 512, (3840,), 3, 16),
    (True, 2049, 1040, (1000, 2000, 1096), 30, 24),
    (True, 4097, 336, (2056,), 1, 128),
    (True, 2100, 640, (2048, 2040), 700, 8),
    (True, 16000, 400, (520,), 64, 64),
]
OTHER = {
    16016: [(False, 5, 272, (520,), 3, 16), (True, 16, 528, (264, 72), 4, 8)],
    16064: [(False, 7, 144, (12312,), 3, 8), (True, 16, 272, (12808,), 4, 16)],
    32016: [(False, 17, 272, (520,), 3, 16), (True, 32, 528, (264, 72), 4, 8)],
    32048: [(False, 31, 144, (12312,), 3, 8), (True, 20, 272, (12808,), 4, 16)],
    48064: [(False, 33, 272, (520,), 3, 16), (True, 48, 528, (264, 7200), 4, 8)],
    64032: [(False, 130, 1040, (520,), 9, 16), (True, 300, 2064, (264, 72), 4, 8)],
    64064: [(False, 50, 272, (8840,), 9, 16), (True, 64, 528, (5128, 4240), 4, 8)],
    64096: [(False, 250, 272, (4104,), 9, 16), (True, 8000, 240, (2056,), 40, 8)],
    128128: [(False, 1000, 1040, (3080,), 40, 16), (True, 1023, 1040, (1544, 1544), 5, 64)],
}
ALL = [(256256, c) for c in LARGE] + [(t, c) for t, cs in OTHER.items() for c in cs]


@pytest.mark.parametrize("tile,case", ALL)
def test_tiles(tile, case):
    fp8, n, k, widths, S, R = case
    print(f"tile {tile} {case}", flush=True)
    args, kw = linear_inputs(n + k, n, k, widths, S, R, fp8, pad=16 if n % 2 else 0)
    check_linear(args, kw, step.lora_linear(*args, **kw), "linear")


BROKEN = {False: (2100, 272, (1992, 2000), 7, 16), True: (2100, 400, (1992, 2000), 7, 16)}
SLOTS = (2200, 272, (2000, 1992), 6, 16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kind", ["none", "one", "runs", "invalid"])
def test_large_tiles_slots(kind, fp8):
    print(f"large tiles slots {kind} fp8={fp8}", flush=True)
    n, k, widths, S, R = SLOTS
    at = torch.arange(n, device="cuda")
    slot = {"none": torch.full_like(at, -1), "one": torch.full_like(at, 4), "runs": at * 5 // n,
            "invalid": torch.where(at % 3 == 0, S + at, at % S)}[kind]
    args, kw = linear_inputs(n, n, k, widths, S, R, fp8, slot=slot)
    check_linear(args, kw, step.lora_linear(*args, **kw), kind)


@pytest.mark.parametrize("fp8", [False, True])
def test_large_tiles_broken_adapter_stays_with_its_rows(fp8):
    n, k, widths, S, R = BROKEN[fp8]
    print(f"large tiles broken adapter fp8={fp8}", flush=True)
    N = sum(widths)
    args, kw = linear_inputs(3, n, k, widths, S, R, fp8, slot=torch.arange(n, device="cuda") % S)
    x, w, a, b, scale, _, slot = args
    y, tol = linear64(args, kw)
    x, a, b = x.clone(), a.clone(), b.clone()
    at = torch.arange(N, device="cuda")[None, :]
    x[1, 5] = math.inf                   # a row of slot 1: all of it, by way of its inner sums
    b[2, 7, 3], b[4, 2500, 0] = math.nan, math.inf
    a[3, 1, 2] = math.nan                # one of the second slice's inner sums
    broken = ((slot == 2)[:, None] & (at == 7)) | ((slot == 4)[:, None] & (at == 2500))
    broken |= (slot == 3)[:, None] & (at >= widths[0])
    broken[1] = True
    got = step.lora_linear(x, w, a, b, scale, widths, slot, **kw)
    assert not got[broken].isfinite().any()
    rest = ~broken & (slot != 3)[:, None]   # (a broken inner sum may reach any column of its row)
    within(got[rest], y[rest], tol[rest], "the others")


@pytest.mark.parametrize("fp8", [False, True])
def test_large_tiles_workspace_and_graph(fp8):
    n, k, widths, S, R = BROKEN[fp8]
    print(f"large tiles graph fp8={fp8}", flush=True)
    N = sum(widths)
    args, kw = linear_inputs(5, n, k, widths, S, R, fp8)
    ws = step.linear_workspace(4 * n, k, 2 * N, len(widths), 2 * R)
    wide = torch.full((n, N + 24), 7.0, device="cuda").bfloat16()
    out = step.lora_linear(*args, out=wide[:, :N], ws=ws, **kw)
    check_linear(args, kw, out, "into wider rows")
    assert (wide[:, N:] == 7).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.lora_linear(*args, out=out, ws=ws, **kw)
        step.lora_linear(*args, out=out, ws=ws, **kw)
    for i in range(4):
        args[0].copy_(randn(gen(40 + i), n, k).bfloat16())
        args[6].copy_(torch.randint(-1, S, (n,), generator=gen(50 + i), device="cuda").int())
        graph.replay()
        torch.cuda.synchronize()
        check_linear(args, kw, out, f"replay {i}")
        assert torch.equal(out, step.lora_linear(*args, ws=ws, **kw))
