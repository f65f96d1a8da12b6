"""The example decoder layer on prompts of one token (GPU): single rows are held to the
element-wise part of the linears' bar."""
import pytest

from test_gpu_decoder_layer import _elements, _prompt_then_token, ex  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts", [(1,), (1, 1, 2)])
def test_prompts_of_one_token(ex, orc, prompts):  # noqa: F811
    _prompt_then_token(ex, orc, prompts, _elements)
