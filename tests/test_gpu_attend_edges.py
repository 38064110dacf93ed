"""Calls of the paged cache's operators at the edge of what they accept: refusals, scales of 0 and NaN, and the
second, careful way of the many-row kernel in every form.  Definition and bounds are those of test_gpu_attend.py."""
import math

import pytest
import torch

from tenant_lora_serving_amd import step
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
