"""Numbers that a C field would cut off (CPU)."""
import pytest

from latent_attention_jagged_b200.binding import _int32


def test_numbers_beyond_32_bits_are_refused():
    _int32(a=0, b=-(1 << 31), c=(1 << 31) - 1)
    for n in (1 << 31, -(1 << 31) - 1, (1 << 32) + 5, 1 << 70):
        with pytest.raises(ValueError, match="budget"):
            _int32(budget=n)
