"""Calls of cross attention that its header rules out and that would read what is not the caller's, refused on the host
before any device work."""
import ctypes as C

import pytest
import torch

from differentiable_gaussian_splatting_dgs_amd import gs, network
from test_attention_host import FAKE, attention


def fwd(a):
    return gs.load_library().gs_attention_fwd(C.byref(a), FAKE, FAKE, FAKE, None, None, None, FAKE, None, FAKE, 1 << 40,
                                              None)


def bwd(a):
    return gs.load_library().gs_attention_bwd(C.byref(a), FAKE, FAKE, FAKE, None, None, None, FAKE, FAKE, FAKE, FAKE,
                                              FAKE, FAKE, FAKE, 1 << 40, None)


@pytest.mark.parametrize("which", ["q", "k", "v", "dout"])
@pytest.mark.parametrize("i", [0, 1, 2])
def test_negative_strides(which, i):
    """Offsets within a tile are unsigned."""
    strides = [1000, 64, 16]
    strides[i] = -strides[i]
    a = attention(**{which + "_stride": (C.c_int64 * 3)(*strides)})
    if which != "dout":
        assert fwd(a) == -1
    assert bwd(a) == -1


def test_negative_mask_stride():
    a = attention(mask_stride=-7)
    assert fwd(a) == -1 and bwd(a) == -1


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_scales_that_overflow_times_log2_e(scale):
    """exp is taken as exp2 of log2 e times the scale: infinity times a logit of 0 would be NaN."""
    a = attention(scale=scale)
    assert fwd(a) == -1 and bwd(a) == -1


@pytest.mark.parametrize("scale", [2.4e38, 1e39, -1e300, float("inf"), float("nan"), 0, 0.0])
def test_scales_from_python(scale, monkeypatch):
    """The framework's error for every scale that the library refuses and for those that no float32 holds."""
    q = torch.zeros(1, 2, 1, 8)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    with pytest.raises(gs.GsError, match="scale"):
        network.cross_attention(q, q, q, scale=scale)
