"""Operands that are no tensors, or no device tensors, are refused with the
binding's own errors, before anything is read from them."""
import numpy as np
import pytest
import torch

import combine_moe_route_topk_amd as moe

CALLS = [("moe_grouped_gemm_mxfp4", 5), ("moe_gather_gemm_mxfp4", 5), ("moe_quantize_mxfp4", 1),
         ("moe_dequant_mxfp4", 2), ("moe_combine_backward", 4)]


@pytest.mark.parametrize("fn,n", CALLS)
@pytest.mark.parametrize("bad", [None, 3, [1, 2], np.zeros((4, 64), np.uint8)])
def test_no_tensor(fn, n, bad):
    with pytest.raises(TypeError, match="must be a tensor"):
        getattr(moe, fn)(*[bad] * n)


@pytest.mark.parametrize("bad", [None, 3])
def test_no_tensor_gradients(bad):
    with pytest.raises(TypeError, match="must be a tensor"):
        moe.moe_dispatch_backward(bad, bad, 2)
    with pytest.raises(TypeError, match="must be a tensor"):
        moe.moe_route_topk_backward(bad, bad, bad, 8)


@pytest.mark.parametrize("fn,n", CALLS)
def test_host_tensor(fn, n):
    with pytest.raises(ValueError, match="device tensor"):
        getattr(moe, fn)(*[torch.zeros((4, 64), dtype=torch.uint8)] * n)
