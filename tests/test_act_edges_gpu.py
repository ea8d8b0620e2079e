"""Calls of the activation operators at the edges of what their contract allows."""
import pytest
import torch

import gradient_compression_amd as gca
import oracle
from tests.gpu_helpers import assert_bitwise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_stochastic_codes_of_values_far_below_their_group(dtype):
    """A draw of 0 rounds every value but 0 away from 0, also one whose quotient by the scale is below
    fp32's smallest number.  Seed 4 draws a 0 for row 20578, column 21 of rows of 32 columns."""
    rows, row, col = 20580, 20578, 21
    for small in (2.0 ** -133, -(2.0 ** -126), 2.0 ** -100, 0.0):
        for top in (126.75 * 2.0 ** 120, 127.0 * 2.0 ** 30, 3.0 * 2.0 ** -120):
            x = torch.zeros(rows, 32)
            x[row, col], x[row, col + 1] = small, top
            x = x.to(dtype)
            want_c, want_e = oracle.act_quant(x.float().numpy(), random=True, seed=4, step=0)
            if small != 0.0 and top > 1.0:
                assert want_c[row, col] == (1 if small > 0 else -1)
            codes = torch.empty(rows, 32, dtype=torch.int8, device="cuda")
            exps = torch.empty(rows, 1, dtype=torch.uint8, device="cuda")
            gca.act_quant(x.cuda(), codes, exps, stochastic=True, seed=4, step=0)
            assert_bitwise(exps, want_e, f"{small} beside {top} exponents")
            assert_bitwise(codes, want_c, f"{small} beside {top} codes")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_weight_gradient_of_no_rows_is_zero_whatever_the_scale(dtype):
    scale = torch.tensor([1.0, -2.0, float("inf"), float("nan"), -float("inf")], device="cuda").repeat(7)
    none = torch.empty(0, 4, dtype=dtype, device="cuda")
    codes = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    exps = torch.empty(0, 2, dtype=torch.uint8, device="cuda")
    dw = torch.full((4, 35), 5.0, device="cuda")
    gca.act_weight_grad(none, codes, exps, dw, col_scale=scale)
    assert bool((dw == 0.0).all())
    dw.fill_(5.0)
    gca.act_weight_grad(none, codes, exps, dw, col_scale=scale, accumulate=True)
    assert bool((dw == 5.0).all())
