"""The example that runs linear attention and the block norms together: training
lowers the loss, and prompts followed by single tokens give what one pass gives."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example():
    path = os.path.join(ROOT, "examples", "linear_attention_block.py")
    spec = importlib.util.spec_from_file_location("linear_attention_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, worst = m.main()
    assert losses[-1] < 0.8 * losses[0]
    # two blocks' bf16 roundings (2^-8 each) on either side, in another order
    assert worst < 4 * 2.0 ** -8
