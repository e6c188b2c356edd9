"""Score options that do not fit the C struct are refused, not cut to 32 bits."""
import pytest

from sparse_mask_transformer_gb300 import build as stof_build
from sparse_mask_transformer_gb300 import stof


@pytest.mark.parametrize("q_start", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1, -(1 << 40)])
def test_a_query_start_past_32_bits(q_start):
    stof_build.build()  # the error's text comes from the library
    with pytest.raises(stof.StofError) as e:
        stof.Score(q_start=q_start).as_c("test", 4)
    assert e.value.status == stof.STOF_ERR_SHAPE
    assert stof.Score(q_start=-(1 << 30)).as_c("test", 4).q_start == -(1 << 30)
