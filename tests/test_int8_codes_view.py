"""Codes written into a view: the zero codes past the columns stay inside it.
(Stand-ins for tensors; nothing is launched.)"""
import pytest
import torch

import mxfp4_quantized_gemm_amd as mx
from tests.test_int8_devices import BF16, F32, I8, Stand


def codes(rows, width, pitch):
    t = Stand(I8, rows, width)
    t.stride = lambda: (pitch, 1)
    t.is_contiguous = lambda: pitch == width
    return t


def pitch_of(monkeypatch, name, rows, cols, c):
    """The codes' pitch that the kernel is given: it writes zero codes from cols
    up to the next multiple of 128 or this pitch, whichever is less."""
    got = []
    monkeypatch.setattr(mx, "_run", lambda fn, args, *a: got.append(args))
    x, s = Stand(BF16, rows, cols), Stand(F32, rows)
    if name == "mxfp4_int8_quantize":
        mx.mxfp4_int8_quantize(x, None, c, s)
    else:
        mx.mxfp4_rmsnorm_int8(x, None, None, 1e-5, None, c, s)
    return got[0][-2]


@pytest.mark.parametrize("name", ["mxfp4_int8_quantize", "mxfp4_rmsnorm_int8"])
def test_zero_codes_stay_inside_the_view(name, monkeypatch):
    ask = lambda *a: pitch_of(monkeypatch, name, *a)
    assert ask(4, 100, codes(4, 100, 100)) == 100   # no zero codes
    assert ask(4, 100, codes(4, 128, 300)) == 300   # up to column 128, the view's end
    assert ask(4, 100, codes(4, 200, 300)) == 300
    assert ask(4, 128, codes(4, 128, 300)) == 300   # a multiple of 128: none
    # the columns past the view are someone else's
    for width, pitch in ((100, 128), (100, 300), (127, 4096)):
        with pytest.raises(ValueError, match="zero codes"):
            ask(4, 100, codes(4, width, pitch))
    # one row has no pitch
    assert ask(1, 100, codes(1, 100, 4096)) == 100
    assert ask(1, 100, codes(1, 110, 4096)) == 110
