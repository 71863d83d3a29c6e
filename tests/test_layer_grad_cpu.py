"""Inputs that require a gradient are refused while autograd records (checked before anything touches a device)."""
from __future__ import annotations

import pytest
import torch

import nvfp4_quantization_group_b200 as hq


def _calls():
    def rows(*shape, grad=False):
        return torch.zeros(shape, dtype=torch.bfloat16, requires_grad=grad)

    i32 = dict(dtype=torch.int32)
    table, lens, slots = torch.zeros((1, 1), **i32), torch.zeros(1, **i32), torch.zeros(1, dtype=torch.int64)
    cache = torch.zeros((2, 1, 1, hq.HQ_KV4_GROUP_BYTES), dtype=torch.uint8)
    rstd, inv = torch.ones(1), torch.zeros(64, dtype=torch.float64)
    x, w, h = rows(1, 128), rows(128), rows(1, 1, 128)
    gx, gw, gh = rows(1, 128, grad=True), rows(128, grad=True), rows(1, 1, 128, grad=True)
    norm, back = hq.add_rmsnorm_fp8_k128, hq.rmsnorm_backward
    return {"norm x": lambda: norm(gx, w), "norm weight": lambda: norm(x, gw), "norm residual": lambda: norm(x, w, gx),
            "norm out": lambda: norm(x, w, x, residual_out=gx), "back dy": lambda: back(gx, x, w, rstd),
            "back h": lambda: back(x, gx, w, rstd), "back dres": lambda: back(x, x, w, rstd, dres=gx),
            "rope q": lambda: hq.rope(gh, None, slots, inv), "rope k": lambda: hq.rope(h, gh, slots, inv),
            "rope out": lambda: hq.rope(h, None, slots, inv, q_out=gh), "append k": lambda: hq.kv4_append(gh, h, slots, cache),
            "append v": lambda: hq.kv4_append(h, gh, slots, cache),
            "attention q": lambda: hq.kv4_attention(gh, cache, table, lens),
            "attention out": lambda: hq.kv4_attention(h, cache, table, lens, out=gh)}


@pytest.mark.parametrize("name", list(_calls()))
def test_refused_while_autograd_records(name):
    call = _calls()[name]
    with pytest.raises(hq.HQError, match="no_grad") as e:
        call()
    assert e.value.status == hq.HQ_ERR_UNSUPPORTED
    # a result that is not a leaf is refused as well, and without recording the call is refused for its device alone
    for mode in (torch.no_grad, torch.inference_mode):
        with mode(), pytest.raises(hq.HQError, match="CUDA device"):
            call()


def test_a_weight_that_requires_a_gradient_may_go_to_the_backward_pass():
    """First derivatives written by hand: the weight is a parameter."""
    x, w = torch.zeros((1, 128), dtype=torch.bfloat16), torch.zeros(128, dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(hq.HQError, match="CUDA device"):
        hq.rmsnorm_backward(x, x, w, torch.ones(1))
