"""norm_rope refuses amax and scale addresses of which one block would read what another writes: the result
would depend on which comes first.  (On the host, before any launch: no GPU needed.)"""
import ctypes

import pytest

from precision_quantized_attention_b200 import _lib

S0 = ctypes.c_void_p(0)
A, B, C, D = 0x20000, 0x20004, 0x20008, 0x2000C


def _status(*tensors):
    """tensors: (codes or not, amax, scale); everything else is as it should be."""
    ios = (_lib.NormRopeIO * len(tensors))()
    for io, (codes, amax, scale) in zip(ios, tensors):
        for k, v in dict(x=0x10000, out=0x100000, amax=amax, scale_out=scale, x_stride_t=256, x_stride_h=128,
                         out_stride_h=2048, out_stride_t=128, H=2, L=16, out_e4m3=codes).items():
            setattr(io, k, v)
    return _lib.load().qattn_norm_rope(ios, len(tensors), 1, 128, 0, 1, 1e-6, 0, S0)


@pytest.mark.parametrize("tensors", [
    [(1, A, A)],                                         # the scale in the place of its amax
    [(1, A, B), (1, B, C)], [(1, B, C), (1, A, B)],      # ... of another tensor's amax
    [(1, A, B), (0, B, None)], [(0, B, None), (1, A, B)],  # ... of a running amax
    [(0, A, None), (1, A, B)], [(1, A, B), (0, A, None)],  # a running amax that is a given one
    [(1, A, B), (0, None, None), (1, C, B)]])            # one scale of two amax
def test_refused(tensors):
    assert _status(*tensors) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("tensors", [
    [(1, A, B), (1, A, B)], [(1, A, B), (1, A, C)], [(0, A, None), (0, A, None)],
    [(1, A, B), (0, C, None), (0, None, None), (1, D, 0x20010)]])
def test_taken(tensors):
    """Past the argument checks: without a GPU the call ends at the device check."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert _status(*tensors) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED)
