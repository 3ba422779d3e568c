"""Limits of the layer operators' arguments, checked on the host before any HIP call (no GPU, no kernel launched)."""
import pytest
import torch

import structured_sparse_gemm_sp24_amd as sp
from tests.test_abi import lib  # noqa: F401
from tests.test_fp8_host import ARG, changed
from tests.test_layer_host import ADAM, T8, T32, Tensor

FP32, FP8 = sp.SP24_FP32, sp.SP24_FP8


@pytest.mark.parametrize("eps", [1e-39, 1e-45, 2.0 ** -127, 2.0 ** -126 * (1 - 2.0 ** -40), -1e-8])
@pytest.mark.parametrize("state", [FP32, FP8])
def test_eps_with_an_infinite_reciprocal_is_refused(lib, state, eps):  # noqa: F811
    """1 / eps passes the largest fp32 below 2^-128: a weight without gradient would become 0 times infinity."""
    one = (Tensor * 1)(Tensor(**(T8 if state == FP8 else T32)))
    assert lib.sp24_adamw(one, *changed(ADAM, state=state, eps=eps)) == ARG


def test_least_eps_is_taken(lib):  # noqa: F811
    """No tensors, so that nothing is launched where there is a device."""
    assert lib.sp24_adamw(None, *changed(ADAM, count=0, eps=2.0 ** -126)) in (sp.SP24_OK, sp.SP24_ERR_DEVICE)


def test_places_in_the_model_are_below_2_to_32():
    p = [torch.zeros(8)] * 2
    for first in (-1, 2 ** 32 - 1, 2 ** 63 - 1):
        with pytest.raises(ValueError, match="first_index"):
            sp.sp24_adamw(p, p, [sp.sp24_adamw_state(x) for x in p], 1, first_index=first)
    with pytest.raises(TypeError):
        sp.sp24_adamw(p, p, [sp.sp24_adamw_state(x) for x in p], 1, first_index=0.5)
    with pytest.raises(ValueError, match="device"):  # a good one: the next check, that of the tensors
        sp.sp24_adamw(p, p, [sp.sp24_adamw_state(x) for x in p], 1, first_index=2 ** 32 - 2)
