"""GPU parity of the 8-bit activation checkpoints with ``oracle/act8.py``:
codes, scales and restored values bit for bit; the backward that reads a
checkpoint against fp64, element by element.

Tolerances (derived, per element): a bf16 rounding is off by at most 2^-8 of
the value.  dA = bf16(sum_i U_i X^_i): the output's rounding, one rounding of
each U, and fp32 accumulation of c terms, each addition off by at most 2^-24
relative of the running sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import multi_refs as M
import oracle_refs as R
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import workloads as WL
from oracle import act8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _bits(t):
    return t.detach().cpu().view(torch.int16).numpy().view(np.uint16)


def _inputs(m, k, seed, kind="normal"):
    X = WL.normal((m, k), 1.0, seed)
    if kind == "spread":            # blocks from 1e-38 to 1e37, some all zero
        e = torch.linspace(-38, 37, (m * k) // 64).view(m, k // 64, 1)
        X = (X.view(m, k // 64, 64) * torch.pow(torch.tensor(10.0), e)).view(m, k)
        X[:, :64] = 0.0
    elif kind == "ties":            # multiples of 1/2 below a block maximum of 127
        X = torch.round(X * 40).clamp(-253, 253) * 0.5
        X[:, ::64] = 127.0
    return WL.bf16(X)


@pytest.mark.parametrize("kind", ["normal", "spread", "ties"])
@pytest.mark.parametrize("mk", [(1, 64), (3, 192), (17, 1088), (257, 4096)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_save_and_restore_bit_exact(mk, kind):
    X = _inputs(*mk, 50 + mk[0], kind)
    act = B.qlora_act_quantize(X.to(DEV))
    Xh = B.qlora_act_dequant(act)
    codes, scale = act8.quantize(R.bf16_to_f64(X))
    assert np.array_equal(act.scale.float().cpu().numpy(), scale)
    assert np.array_equal(act.codes.cpu().numpy(), codes)
    assert np.array_equal(_bits(Xh), act8.dequant_bits(codes, scale))


def test_save_writes_nothing_past_the_end():
    m, k = 5, 192
    X = _inputs(m, k, 3).to(DEV)
    codes = torch.full((m * k + 256,), 77, dtype=torch.int8, device=DEV)
    scale = torch.full((m * k // 64 + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    act = B.Act8(codes[:m * k].view(m, k), scale[:m * k // 64].view(m, k // 64), m, k)
    B.qlora_act_quantize(X, out=act)
    out = torch.full((m * k + 256,), 5.0, dtype=torch.bfloat16, device=DEV)
    B.qlora_act_dequant(act, out=out[:m * k].view(m, k))
    torch.cuda.synchronize()
    assert bool((codes[m * k:] == 77).all()) and bool((scale[m * k // 64:] == 3.0).all())
    assert bool((out[m * k:] == 5.0).all())


def test_empty_checkpoint():
    act = B.qlora_act_quantize(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV))
    assert B.qlora_act_dequant(act).shape == (0, 128)


@pytest.mark.parametrize("r", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("mnk", [(1, 72, 64), (17, 520, 192), (64, 264, 128), (300, 264, 1088), (1100, 72, 4160)],
                         ids=lambda s: f"m{s[0]}_n{s[1]}_k{s[2]}")
def test_backward_from_a_checkpoint(mnk, r):
    m, n, k = mnk
    c = M.case(m, n, k, r, 1, "one", 900 + m + r)
    act = B.qlora_act_quantize(c.X.to(DEV))
    T = WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float())
    dX, dA, dB = B.qlora_linear_bwd_act8(c.dY.to(DEV), act, c.weight(DEV), c.A[0].to(DEV), c.B[0].to(DEV), r,
                                         float(c.s[0]), T.to(DEV))
    codes, scale = act8.quantize(c.Xf)
    c.check_bwd((dX, dA[None], dB[None]), act8.dequant_values(codes, scale), R.bf16_to_f64(T))
    assert B.qlora_poll_device_error() == 0


def test_gradient_follows_the_restored_input_and_is_the_same_twice():
    """dA of the checkpoint is dA of the restored X through the ordinary
    backward up to accumulation order; two runs agree bit for bit."""
    m, n, k, r = 513, 264, 1088, 32
    c = M.case(m, n, k, r, 1, "one", 77)
    act = B.qlora_act_quantize(c.X.to(DEV))
    Xh = B.qlora_act_dequant(act)
    args = (c.weight(DEV), c.A[0].to(DEV), c.B[0].to(DEV), r, float(c.s[0]))
    T = WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float()).to(DEV)
    a = B.qlora_linear_bwd_act8(c.dY.to(DEV), act, *args, T)
    b = B.qlora_linear_bwd_act8(c.dY.to(DEV), act, *args, T)
    ref = B.qlora_linear_bwd(c.dY.to(DEV), Xh, *args, T=T)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(a[0], ref[0]) and torch.equal(a[2], ref[2])
    d = (a[1].float() - ref[1].float()).abs()
    assert bool((d <= 2.0 ** -7 * ref[1].float().abs() + 1e-3 * float(ref[1].float().abs().max())).all())


def test_backward_of_an_empty_batch_writes_zeros():
    c = M.case(1, 72, 64, 16, 1, "one", 5)
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    act = B.qlora_act_quantize(empty)
    dX, dA, dB = B.qlora_linear_bwd_act8(torch.empty(0, 72, dtype=torch.bfloat16, device=DEV), act, c.weight(DEV),
                                         c.A[0].to(DEV), c.B[0].to(DEV), 16, 1.0,
                                         torch.empty(0, 16, dtype=torch.bfloat16, device=DEV))
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()
