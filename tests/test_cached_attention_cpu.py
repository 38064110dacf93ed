"""What decode_step's CachedAttention refuses before anything is launched (no GPU)."""
import pytest

from tenant_lora_serving_amd.decode_step import CachedAttention


def make(context=20, prefixes=(40, 7), page=16):
    return CachedAttention(4, 2, 64, 3, context, prefixes, page=page, device="cpu")


def test_sizes_of_the_cache():
    for bad in (dict(context=0), dict(context=-3), dict(prefixes=(5, -1)), dict(page=0)):
        with pytest.raises(ValueError):
            make(**bad)
    a = make(prefixes=(0, 3))
    assert a.prefix.lens.tolist() == [0, 3] and a.prefix.pages.shape == (2, 1)
