"""Moves of a module between types and devices."""
import copy

import pytest
import torch

import multi_refs as M
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import layer as L

DEV = "cuda:0"


def _module():
    scale = torch.tensor([16 / 48, 0.1, 2.0])
    return L.MultiQLoRALinear(B.NF4Weight(None, None, None, 24, 64), torch.zeros(3, 16, 64), torch.zeros(3, 24, 16),
                              scale), scale


@pytest.mark.parametrize("move", [lambda m: m.bfloat16(), lambda m: m.to(torch.bfloat16), lambda m: m.to(dtype=torch.bfloat16, device="cpu"),
                                  lambda m: torch.nn.Sequential(m).bfloat16()[0], lambda m: copy.deepcopy(m).bfloat16()])
def test_scales_stay_fp32_in_a_bf16_model(move):
    """The scales are fp32 numbers of the calls, like the one-adapter layer's, not parameters of the model's type."""
    m, scale = _module()
    m = move(m)
    assert m.A.dtype == torch.bfloat16 and m.scale.dtype == torch.float32 and torch.equal(m.scale, scale)
    assert set(m.state_dict()) == {"A", "B", "scale"} and "scale" in dict(m.named_buffers())


def test_scales_move_with_the_module():
    m, scale = _module()
    m.to("meta", torch.bfloat16)
    assert m.scale.device.type == "meta" and m.scale.dtype == torch.float32


@pytest.mark.gpu
def test_a_bf16_model_gives_what_it_gave():
    c = M.case(40, 264, 192, 16, 3, "mixed", 15000)
    m = L.MultiQLoRALinear(c.weight(DEV), c.A, c.B, torch.tensor([16 / 48, 0.1, 2.0])).to(DEV)
    X, ids = c.X.to(DEV), c.ids.to(DEV)
    with torch.no_grad():
        want = m(X, ids)
        assert torch.equal(m.to(torch.bfloat16)(X, ids), want)
