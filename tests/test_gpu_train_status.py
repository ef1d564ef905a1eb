"""The training example reports an error of any of its steps, not the last one's alone."""

import os
import sys

import pytest
import torch

import moe_expert_layer_ep_gb300 as M

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import train_experts as X  # noqa: E402

pytestmark = pytest.mark.gpu


def test_an_id_out_of_range_in_the_first_step_is_reported(monkeypatch):
    route, seen = M.moe_route, []

    def bad_first(*args, **kwargs):
        ids, weights, logits = route(*args, **kwargs)
        if not seen:
            ids[3, 1] = 77
        seen.append(ids)
        return ids, weights, logits

    monkeypatch.setattr(M, "moe_route", bad_first)
    with pytest.raises(RuntimeError, match="MOE_ERR_EXPERT_ID"):
        X.train(steps=4)
    assert len(seen) == 4


def test_an_error_of_a_product_in_the_first_step_is_reported(monkeypatch):
    product, seen = M.moe_expert_gemm_dgrad, []

    def bad_first(dy, w, start, counts, status, **kwargs):
        if not seen:
            counts = counts.clone()
            counts[-1] = dy.shape[0] + 1   # an expert that does not fit: it is left out
        seen.append(counts)
        return product(dy, w, start, counts, status, **kwargs)

    monkeypatch.setattr(M, "moe_expert_gemm_dgrad", bad_first)
    with pytest.raises(RuntimeError, match="MOE_ERR_INVALID_ARG"):
        X.train(steps=3)
    assert len(seen) == 3


def test_steps_without_an_error_report_none():
    assert all(torch.isfinite(torch.tensor(X.train(steps=2))))
