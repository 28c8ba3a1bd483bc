"""The feed-forward example end to end: its training loss falls through the
norm's gradient, and the 8-bit block stays near the trained weights."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_feed_forward_example():
    path = os.path.join(ROOT, "examples", "feed_forward_int8.py")
    spec = importlib.util.spec_from_file_location("feed_forward_int8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, far = m.main(["--hidden", "512", "--inner", "1024", "--tokens", "256", "--steps", "12"])
    assert losses[-1] < losses[0]
    # Codes are off by at most half a step of 1 / 127 of the row's largest
    # value, under 2 % of a typical one, in each of the four operands; the
    # products' terms add up at random.
    assert all(0 < v < 0.05 for v in far.values()), far
