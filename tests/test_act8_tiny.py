"""How far a checkpoint of very small values is off: blocks whose c / 127 is a
normal bf16 number keep the bound of half a step; below, where it has few bits,
values stay within 2 c."""
import numpy as np
import pytest
import torch

from bit_nf4_quantized_qlora_b200 import binding as B
from oracle import act8, quant


def _blocks(low, high, seed):
    """[4096 x 64] bf16 values whose blocks' largest magnitudes lie between 2^low and 2^high."""
    g = np.random.default_rng(seed)
    c = np.exp2(g.uniform(low, high, size=(4096, 1)))
    x = g.uniform(-1.0, 1.0, size=(4096, 64)) * c
    x[:, 0] = c[:, 0]
    return quant.bf16_bits_to_f32(quant.bf16_rne_bits(x.astype(np.float32)))


def _check_bound(X):
    x = X.astype(np.float64)
    codes, scale = act8.quantize(x)
    Xh, step = act8.dequant_values(codes, scale), np.repeat(scale.astype(np.float64), 64, axis=1)
    # One rounding: half a step, 2^-8 of the value or half the smallest subnormal, 2^-134.
    off = np.abs(Xh - x) - (0.5 * step + np.maximum(2.0 ** -8 * np.abs(Xh), 2.0 ** -134))
    return off.max(), np.abs(Xh).max(1) / np.abs(x).max(1)


def test_half_a_step_down_to_two_to_the_minus_119():
    for low, high in ((-119.0, -118.0), (-119.0, -90.0)):
        off, _ = _check_bound(_blocks(low, high, 1))
        assert off <= 0


def test_below_it_the_step_is_coarse_and_values_stay_within_twice_the_largest():
    X = _blocks(-133.0, -119.1, 2)
    X = X[np.abs(X).max(1) > 0]
    off, grown = _check_bound(X)
    assert off > 0                                    # so the bound cannot be promised here
    assert grown.max() <= 2.0


@pytest.mark.gpu
@pytest.mark.parametrize("low,high", [(-119.0, -90.0), (-133.0, -119.0)])
def test_tiny_blocks_on_the_gpu_are_the_oracles(low, high):
    X = _blocks(low, high, 3)
    codes, scale = act8.quantize(X.astype(np.float64))
    act = B.qlora_act_quantize(torch.from_numpy(X).to(torch.bfloat16).cuda())
    assert np.array_equal(act.codes.cpu().numpy(), codes)
    assert np.array_equal(act.scale.float().cpu().numpy(), scale)
    bits = B.qlora_act_dequant(act).cpu().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(bits, act8.dequant_bits(codes, scale))
