"""CPU: arguments of the E4M3 operators that a call does not need (meta tensors, nothing reaches the library)."""
import pytest
import torch

import block_scaled_fp4_e2m1_amd as bs
from test_block_ops_refusals import reaches_device_check, refused
from test_fp8_refusals import f, i, m, q


@pytest.mark.parametrize("epilogue,more,good,bad", [
    (bs.MOE_STORE_BF16, {}, {"out": m(9, 256)}, {"out_q": q(9, 128), "out_s": f(1, 9)}),
    (bs.MOE_SILU_MUL_QUANT, {}, {"out_q": q(9, 128), "out_s": f(1, 9)}, {"out": m(9, 256)}),
    (bs.MOE_WEIGHTED_COMBINE, {"row_of": i(3, 3), "topk_weights": f(3, 3)}, {"out": m(3, 256)}, {"out_q": q(9, 128), "out_s": f(1, 9)})])
def test_grouped_outputs_that_are_not_written(epilogue, more, good, bad):
    """A given output would come back as it was."""
    args = (q(9, 272), f(3, 9), i(5), q(4, 256, 272), f(4, 2, 3), epilogue)
    reaches_device_check(bs.fp8_moe_grouped_gemm, *args, **more, **good)
    for name, t in bad.items():
        refused(f"{name} is not written", bs.fp8_moe_grouped_gemm, *args, **more, **{name: t})
        refused(f"{name} is not written", bs.fp8_moe_grouped_gemm, *args, **more, **good, **{name: t})


def test_linear_backward_without_what_it_does_not_read():
    dy, x, WT, SWT = m(5, 144), m(5, 272), q(272, 144), f(3, 2)
    b = bs.fp8_linear_backward
    reaches_device_check(b, dy, None, WT, SWT, need_dW=False)
    reaches_device_check(b, dy, x, None, None, need_dx=False)
    reaches_device_check(b, dy, None, None, None, need_dx=False, need_dW=False)
    refused("dW needs x", b, dy, None, WT, SWT)
    refused("dx needs WT and SWT", b, dy, x, None, SWT)
    refused("dx needs WT and SWT", b, dy, x, WT, None)
    # what is given all the same is held to its shape
    refused("dy has 5 rows but x has 6", b, dy, m(6, 272), WT, SWT, need_dW=False)
    refused("WT must have", b, dy, x, q(144, 272), SWT, need_dx=False)
    refused("SWT must have", b, dy, None, WT, f(2, 3), need_dW=False)
    refused("multiple of 16", b, dy, None, q(264, 144), f(3, 2), need_dW=False)
    refused("dW_dtype", b, dy, x, WT, SWT, dW_dtype=torch.float16)
