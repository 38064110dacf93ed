"""What decode_step's CachedAttention refuses before anything is launched (no GPU)."""
import subprocess
import sys

import pytest
import torch

from tenant_lora_serving_amd.decode_step import CachedAttention


def make(context=20, prefixes=(40, 7), page=16):
    return CachedAttention(4, 2, 64, 3, context, prefixes, page=page, device="cpu")


def projected(n):
    return torch.zeros(n, (4 + 2 * 2) * 64, dtype=torch.bfloat16)


@pytest.mark.parametrize("i,n", [(0, 41), (0, 39), (0, 0), (0, 500), (1, 8), (1, 48), (1, 100)])
def test_a_prefix_has_the_length_that_it_was_made_with(i, n):
    """More tokens than its pages hold would index past the table on the device, fewer leave zeros behind them."""
    with pytest.raises(ValueError, match="prefix"):
        make().fill_prefix(i, projected(n))


def test_no_such_prefix():
    for a, i in ((make(), 2), (make(prefixes=()), 0), (make(), -1)):
        with pytest.raises(IndexError):
            a.fill_prefix(i, projected(7))


def test_sizes_of_the_cache():
    for bad in (dict(context=0), dict(context=-3), dict(prefixes=(5, -1)), dict(page=0)):
        with pytest.raises(ValueError):
            make(**bad)
    a = make(prefixes=(0, 3))
    assert a.prefix.lens.tolist() == [0, 3] and a.prefix.pages.shape == (2, 1)


def test_the_command_refuses_a_prefix_without_a_context():
    for more in (["--prefix", "50"], ["--context", "-1"], ["--context", "9", "--prefix", "-2"]):
        r = subprocess.run([sys.executable, "-m", "tenant_lora_serving_amd.decode_step", "--rows", "3", *more],
                           capture_output=True, text=True, timeout=100)
        assert r.returncode == 2 and "--" in r.stderr, r.stderr[-500:]
