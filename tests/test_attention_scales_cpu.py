"""Which scales the attention entry points accept: no GPU."""
import pytest

from test_attention_cpu import EDEVICE, EINVAL, call, no_gpu

ATTENTION = ("pq2_attention_paged", "pq2_attention_prompt")


@pytest.mark.parametrize("name", ATTENTION)
@pytest.mark.parametrize("scale", [2.36e38, 3.4e38])
def test_scales_beyond_fp32_times_log2e(name, scale):
    """They would make scores of zero NaN."""
    assert call(name, scale=scale) == EINVAL


@no_gpu
@pytest.mark.parametrize("name", ATTENTION)
@pytest.mark.parametrize("scale", [1.4e-45, 1.0, 2.35e38])
def test_scales_from_the_smallest_to_the_largest(name, scale):
    assert call(name, scale=scale) == EDEVICE
