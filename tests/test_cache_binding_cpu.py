"""The binding of the paged cache's operators (step.py) over a host-only build of their entry points: what reaches
the library, and which calls are refused.  The tensors are the host's and pass for a device's."""
import pytest
import torch

from tenant_lora_serving_amd import step
from tenant_lora_serving_amd.lora import LoraError
from test_attend_host_cpu import FEW, L, launches, reset  # noqa: F401


class OnDevice(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 0


def dev(t):
    return t.as_subclass(OnDevice)


@pytest.fixture(autouse=True)
def host(L, monkeypatch):  # noqa: F811
    L.step_status_string = step.lib().step_status_string
    monkeypatch.setattr(step, "_lib", L)
    monkeypatch.setattr(step, "_raw_stream", lambda d: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)


def ints(v):
    return dev(torch.tensor(v, dtype=torch.int32))


B, COLS = 4, 7
CACHE = dev(torch.zeros(9, 16, 2, 64, dtype=torch.bfloat16))
Q = dev(torch.zeros(B, 8, 64, dtype=torch.bfloat16))
WS = dev(torch.zeros(1 << 26, dtype=torch.uint8))
TABLE = ints([[7 * b + i for i in range(COLS)] for b in range(B)])


def attend(**kw):
    a = dict(pages=TABLE, lens=ints([100] * B), ws=WS)
    a.update(kw)
    return step.paged_attention(Q, CACHE, CACHE, a.pop("pages"), a.pop("lens"), **a)


def prefix(pages):
    return step.Prefixes(pages, ints([50] * B), ints(list(range(B + 1))))


# Rows of a table that lie on one another: one row for all requests, a window that slides, one column for all.
OVERLAPPING = [TABLE[:1].expand(B, -1), ints(list(range(2 * COLS))).as_strided((B, COLS), (1, 1)), ints([[3]]).expand(B, 1)]


def test_tables_pass_with_their_strides(L):  # noqa: F811
    wide = ints([[0] * 20] * B)
    for pages in (TABLE, wide[:, 3:3 + COLS], TABLE[:, :1], TABLE[:, :0], ints([[]] * B)):
        attend(pages=pages)
        attend(prefix=prefix(pages))
    assert step._table(wide[:, 3:3 + COLS], "pages", B, 0) == (wide.data_ptr() + 12, 20, COLS)
    assert [x[0] for x in launches(L)][0] == FEW


@pytest.mark.parametrize("pages", OVERLAPPING, ids=["one row", "window", "one column"])
def test_tables_whose_rows_overlap_are_refused(L, pages):  # noqa: F811
    assert step._table(pages, "pages", B, 0)[1] == pages.stride(0)
    with pytest.raises(LoraError):
        attend(pages=pages)
    with pytest.raises(LoraError):
        attend(prefix=prefix(pages))
    assert launches(L) == []


def test_one_request_of_an_expanded_table(L):  # noqa: F811
    """A single row's stride means nothing."""
    step.paged_attention(Q[:1], CACHE, CACHE, TABLE[:1].expand(1, -1), ints([100]), ws=WS)
    assert len(launches(L)) == 1
