"""rope_table refuses sizes that do not fit the C call's 32 bits before anything is
allocated: cut down to 32 bits they would name another, valid table."""
import pytest

from exact_attention_154_b200 import fa


@pytest.mark.parametrize("kw", [dict(max_pos=2 ** 32 + 8), dict(max_pos=2 ** 31), dict(rot=2 ** 32 + 64),
                                dict(original_max_pos=2 ** 32 + 4096), dict(original_max_pos=2 ** 31),
                                dict(original_max_pos=-2 ** 32 + 4096), dict(rot=2 ** 70)])
def test_sizes_beyond_32_bits(kw):
    args = dict(max_pos=8, rot=64, scaling="yarn", factor=4.0, original_max_pos=4096)
    args.update(kw)
    with pytest.raises(ValueError, match="32 bits"):
        fa.rope_table(**args)
