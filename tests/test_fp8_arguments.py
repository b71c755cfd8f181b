"""CPU: arguments of the E4M3 operators that a call does not need (meta tensors, nothing reaches the library)."""
import pytest

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
