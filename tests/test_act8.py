"""8-bit activation checkpoints on the CPU: pins of ``oracle/act8.py``, and the
entry points' argument checks (every call returns before the library's first
CUDA call)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from bit_nf4_quantized_qlora_b200 import binding as B
from oracle import act8, quant

P = 0x10000000
MIS = P + 8


def _bf16(a):
    return quant.bf16_bits_to_f32(quant.bf16_rne_bits(np.asarray(a, dtype=np.float32))).astype(np.float64)


def _rint_half_even(f: Fraction) -> int:
    return round(f)      # Python rounds a Fraction's halves to even


def test_codes_by_exact_rational_arithmetic():
    """Brute force: the code of every element from the exact quotient."""
    rng = np.random.default_rng(1)
    X = _bf16(rng.standard_normal((3, 128)) * np.array([[1.0], [1e-20], [300.0]]))
    codes, scale = act8.quantize(X)
    for i in range(3):
        for j in range(128):
            s = Fraction(float(scale[i, j // 64]))
            want = max(-127, min(127, _rint_half_even(Fraction(float(X[i, j])) / s)))
            assert codes[i, j] == want, (i, j)


def test_ties_go_to_the_even_code():
    """scale is exactly 1 (c = 127); quotients on half integers."""
    X = np.zeros((1, 64))
    X[0, :6] = [127.0, 0.5, 1.5, 2.5, -0.5, -1.5]
    codes, scale = act8.quantize(X)
    assert scale[0, 0] == 1.0
    assert list(codes[0, :6]) == [127, 0, 2, 2, 0, -2]


def test_zero_and_tiny_blocks():
    X = np.zeros((2, 64))
    X[1, 3] = _bf16([3e-39])[0]          # bf16 subnormal: c / 127 keeps few bits or none
    codes, scale = act8.quantize(X)
    assert scale[0, 0] == 0.0 and not codes[0].any()
    assert np.all(np.abs(codes) <= 127)
    assert not act8.dequant_values(codes, scale)[0].any()


def test_error_is_half_a_step_plus_one_rounding():
    rng = np.random.default_rng(2)
    X = _bf16(rng.standard_normal((64, 256)) * np.exp(rng.standard_normal((64, 1)) * 4))
    codes, scale = act8.quantize(X)
    Xh = act8.dequant_values(codes, scale)
    step = np.repeat(scale.astype(np.float64), 64, axis=1)
    # A scale rounded down lets the largest quotient reach 127 (1 + 2^-8) =
    # 127.496, still within half a step of 127.
    assert np.all(np.abs(Xh - X) <= 0.5 * step + 2.0 ** -8 * np.abs(Xh))


def test_lossless_when_the_block_lies_on_its_grid():
    rng = np.random.default_rng(3)
    q = rng.integers(-127, 128, size=(4, 64))
    q[:, 0] = 127
    X = q * 0.25
    codes, scale = act8.quantize(X)
    assert np.array_equal(codes, q) and np.array_equal(act8.dequant_values(codes, scale), X)


# ---- argument checks --------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def _act(m=16, k=128, codes=P, scale=P):
    return B.Act8C(codes, scale, m, k)


def test_struct_layout():
    assert ctypes.sizeof(B.Act8C) == 32
    assert ctypes.sizeof(B.AdapterSetC) == 32


def test_quantize_and_dequant_reject_bad_arguments(lib):
    q = lambda **a: lib.qlora_act_quantize(a.get("X", P), a.get("m", 16), a.get("k", 128), a.get("c", P),
                                           a.get("s", P), None)
    assert q(X=None) == q(c=None) == q(s=None) == B.QLORA_ERR_NULL
    assert q(X=MIS) == q(c=MIS) == q(s=MIS) == B.QLORA_ERR_ALIGN
    assert q(k=100) == q(k=0) == q(m=-1) == q(m=1 << 31, k=1 << 31) == B.QLORA_ERR_SHAPE
    assert q(m=0, X=None, c=None, s=None) == B.QLORA_OK
    d = lambda a, X=P: lib.qlora_act_dequant(ctypes.byref(a) if a else None, X, None)
    assert d(None) == d(_act(codes=0)) == d(_act(scale=0)) == d(_act(), X=None) == B.QLORA_ERR_NULL
    assert d(_act(codes=MIS)) == d(_act(), X=MIS) == B.QLORA_ERR_ALIGN
    assert d(_act(k=96)) == d(_act(m=-1)) == B.QLORA_ERR_SHAPE
    assert d(_act(m=0), X=None) == B.QLORA_OK


def test_bwd_act8_rejects_bad_arguments(lib):
    w = B.NF4WeightC(P, P, P, 1024, 1024, 64, 256)

    def f(act=_act(16, 1024), **a):
        return lib.qlora_linear_bwd_act8(a.get("dY", P), ctypes.byref(act) if act else None, a.get("T", P),
                                         a.get("m", 16), ctypes.byref(w), a.get("A", P), a.get("B", P), a.get("r", 16),
                                         2.0, a.get("dX", P), a.get("dA", P), a.get("dB", P), a.get("ws", P),
                                         a.get("ws_bytes", 1 << 20), None)

    assert f(act=None) == f(T=None) == f(dY=None) == f(dA=None) == f(A=None) == B.QLORA_ERR_NULL
    assert f(act=_act(16, 1024, codes=0)) == B.QLORA_ERR_NULL
    assert f(act=_act(15, 1024)) == f(act=_act(16, 512)) == f(r=24) == f(r=0) == f(m=-1) == B.QLORA_ERR_SHAPE
    assert f(act=_act(16, 1024, scale=MIS)) == f(T=MIS) == f(dX=MIS) == B.QLORA_ERR_ALIGN
    assert f(ws=None) == f(ws_bytes=100) == B.QLORA_ERR_WORKSPACE


def test_binding_refuses_what_it_cannot_pass_on():
    """The Python calls look at tensors before the library does."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.qlora_act_quantize(x)
    with pytest.raises(ValueError, match="multiple of 64"):
        B.qlora_act_quantize(torch.zeros(4, 100, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        B.qlora_act_dequant(B.Act8.empty(4, 128, "cpu"))
