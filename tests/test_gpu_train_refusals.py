"""Arguments of the training operators that are no matrices are refused as such."""

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

pytestmark = pytest.mark.gpu


def _cases():
    bf = torch.bfloat16
    m, w = torch.zeros((128, 64), dtype=bf, device="cuda"), torch.zeros((1, 64, 64), dtype=bf, device="cuda")
    at = [torch.tensor([v], dtype=torch.int32, device="cuda") for v in (0, 128)] + [torch.zeros(4, dtype=torch.int32, device="cuda")]
    dst = torch.arange(128, dtype=torch.int32, device="cuda").view(128, 1)
    wt = torch.ones((128, 1), device="cuda")
    gu, w13 = torch.zeros((128, 128), dtype=bf, device="cuda"), torch.zeros((1, 128, 64), dtype=bf, device="cuda")
    return {
        "sort.x": lambda t: M.moe_sort_tokens(t, dst, rows=128),
        "sort.out": lambda t: M.moe_sort_tokens(m, dst, out=t),
        "unsort.y": lambda t: M.moe_unsort_tokens(t, dst),
        "unsort.out": lambda t: M.moe_unsort_tokens(m, dst, out=t),
        "unsort_backward.dout": lambda t: M.moe_unsort_tokens_backward(t, m, dst, wt),
        "unsort_backward.y": lambda t: M.moe_unsort_tokens_backward(m, t, dst, wt),
        "unsort_backward.dy": lambda t: M.moe_unsort_tokens_backward(m, m, dst, wt, dy=t),
        "gemm.x": lambda t: M.moe_expert_gemm(t, w, *at),
        "gemm.y": lambda t: M.moe_expert_gemm(m, w, *at, y=t),
        "swiglu.x": lambda t: M.moe_expert_gemm_swiglu(t, w13, *at),
        "swiglu.h": lambda t: M.moe_expert_gemm_swiglu(m, w13, *at, h=t),
        "swiglu.gu": lambda t: M.moe_expert_gemm_swiglu(m, w13, *at, gu=t),
        "dgrad.dy": lambda t: M.moe_expert_gemm_dgrad(t, w, *at),
        "dgrad.dx": lambda t: M.moe_expert_gemm_dgrad(m, w, *at, dx=t),
        "dgrad_swiglu.dy": lambda t: M.moe_expert_gemm_dgrad_swiglu(t, w, gu, *at),
        "dgrad_swiglu.gu": lambda t: M.moe_expert_gemm_dgrad_swiglu(m, w, t, *at),
        "dgrad_swiglu.dgu": lambda t: M.moe_expert_gemm_dgrad_swiglu(m, w, gu, *at, dgu=t),
        "wgrad.dy": lambda t: M.moe_expert_gemm_wgrad(t, m, *at),
        "wgrad.x": lambda t: M.moe_expert_gemm_wgrad(m, t, *at),
    }


NAMES = ("sort.x sort.out unsort.y unsort.out unsort_backward.dout unsort_backward.y unsort_backward.dy gemm.x gemm.y "
         "swiglu.x swiglu.h swiglu.gu dgrad.dy dgrad.dx dgrad_swiglu.dy dgrad_swiglu.gu dgrad_swiglu.dgu wgrad.dy "
         "wgrad.x").split()


@pytest.mark.parametrize("name", NAMES)
def test_a_vector_a_number_or_a_cube_in_place_of_a_matrix(name):
    call = _cases()[name]
    for shape in ((64,), (), (2, 64, 64)):
        with pytest.raises(ValueError):
            call(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
