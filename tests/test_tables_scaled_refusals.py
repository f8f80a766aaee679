"""build_tables_scaled without a GPU: what it refuses before it touches a device."""
import pytest

import rotary_position_embedding_rope_gb300 as R


@pytest.mark.parametrize("kind", ["linear", "yarn"])
@pytest.mark.parametrize("zero", [0, 0.0, -0.0])
def test_a_factor_of_zero_is_not_the_default(kind, zero):
    with pytest.raises(ValueError, match="value_scale"):
        R.build_tables_scaled(kind, 64, 4, 2.0, 128, value_scale=zero)
