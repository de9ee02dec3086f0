"""The example layer runs: prompts, then single tokens in a replayed graph, against the whole."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def _example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "softmax_layer", os.path.join(root, "examples", "softmax_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("argv", [
    ["--heads", "4", "--kv-heads", "2", "--dim", "64", "--prompts", "70,3,1,129", "--new", "5"],
    ["--heads", "32", "--kv-heads", "8", "--dim", "128", "--prompts", "200,31", "--new", "3"],
])
def test_tokens_one_at_a_time_are_the_whole(argv):
    """A block that grows keeps the larger scale, so a token may be rounded twice, by 2^-4 of its
    block's smallest kept digits at most; the outputs are averages over many: a tenth of that."""
    off, all_free = _example().main(argv)
    assert all_free
    assert off < 2.0 ** -4
