"""The example of a decoder layer's attention half, as a user runs it."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_decode_layer():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # queries and outputs are rounded to binary16 (2^-11 at most each, of scores a few units wide)
    assert example.main(["--batch", "3", "--prompt", "700", "--steps", "6"]) < 2e-3
