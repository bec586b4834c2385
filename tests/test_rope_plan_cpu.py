"""Plans of the rope at the ends of their arguments.  CPU only."""
import pytest

import deepseek_sparse_attention_gb300 as dsa


@pytest.mark.parametrize("magnitude", [3.5e38, -1e39, 1e300])
def test_a_magnitude_beyond_float32_is_refused(magnitude):
    """It would be infinite in the plan, and every result infinite or NaN."""
    with pytest.raises(dsa.DsaError):
        dsa.make_rope(64, 1e4, magnitude=magnitude)


@pytest.mark.parametrize("magnitude", [3.4e38, -1.0, 0.0])
def test_a_magnitude_of_float32_is_kept(magnitude):
    assert dsa.make_rope(64, 1e4, magnitude=magnitude).magnitude == pytest.approx(magnitude, rel=2.0 ** -24)
