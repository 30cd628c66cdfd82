"""Infinities and NaN where a row has them: they reach what the formulas say
they reach, with the formulas' signs, and nothing else."""
import numpy as np
import pytest
import torch

import multi_refs as M
import oracle_refs as R
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import workloads as WL

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _same_kind(got, ref):
    """Finite, +inf, -inf or NaN alike, element by element."""
    g = R.bf16_to_f64(got)
    assert g.shape == ref.shape
    for kind in (np.isnan, np.isposinf, np.isneginf):
        bad = kind(g) != kind(ref)
        assert not bad.any(), f"{kind.__name__}: {bad.sum()} elements, {kind(g).sum()} for {kind(ref).sum()}"


def _ids(m, count, order):
    """Every adapter's last slot of 64 rows has pad rows, the first of them with an infinite last row."""
    ids = np.arange(m) * count // m if order == "runs" else np.arange(m) * 7 % count
    return torch.from_numpy(ids.astype(np.int32))


@pytest.mark.parametrize("what", ["X", "dY", "T"])
@pytest.mark.parametrize("order", ["runs", "mixed"])
@pytest.mark.parametrize("m,count", [(1, 1), (5, 2), (70, 1), (130, 3), (600, 4)])
def test_an_infinity_in_an_adapters_last_row(m, count, order, what):
    """The pad rows of a group's last slot repeat that row."""
    n, k, r = 72, 192, 16
    c = M.case(m, n, k, r, count, "one", 14000 + m)
    ids = _ids(m, count, order)
    rows = np.nonzero(ids.numpy() == 0)[0]
    assert len(rows) % 16
    T = WL.bf16(WL.normal((m, r), 1.0, 14001))
    {"X": c.X, "dY": c.dY, "T": T}[what][rows[-1], 3] = float("-inf")
    c = M.Case(c.W, c.X, c.dY, c.A, c.B, c.scale, ids)
    A, Bm, s, idd = c.on(DEV)
    got = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), c.weight(DEV), A, Bm, s, idd, T=T.to(DEV))
    with np.errstate(invalid="ignore"):
        want = M.multi.bwd(c.dYf, c.Xf, R.bf16_to_f64(T), c.W_hat(), c.Af, c.Bf, c.s, c.ids_np)
    for g, w in zip(got[1:], want[1:]):
        _same_kind(g, w)


@pytest.mark.parametrize("dq", [B.QLORA_DQ_LINEAR8, B.QLORA_DQ_FP8_MEAN])
@pytest.mark.parametrize("k", [192, 320, 1024, 1280])          # the streaming kernel's three forms
@pytest.mark.parametrize("m", [1, 3, 4, 5, 16])
def test_infinite_activations_of_a_decode_batch(m, k, dq):
    """Y of a row with infinities has the infinities and NaN of X . W^T: signs
    by the weights, NaN where a weight is zero or two infinities cancel.  The
    other rows are what they are without them."""
    n, r, count = 264, 16, 3
    c = M.case(m, n, k, r, count, "none", 14100 + m + k)
    c.W[5, :] = 0.0                                   # a row of zero blocks
    c.W[:, 70] = 0.0                                  # a column of zero codes
    ids = torch.arange(m, dtype=torch.int32) % (count + 1)
    A, Bm, s = (t.to(DEV) for t in (c.A, c.B, c.scale))
    w = B.qlora_quantize_4bit_dq(c.W.to(DEV), B.QLORA_CODEBOOK_NF4, dq_format=dq)
    W = R.bf16_to_f64(B.qlora_dequant(w))
    clean = B.qlora_linear_fwd_multi(c.X.to(DEV), w, A, Bm, s, ids.to(DEV))
    inf, nan = float("inf"), float("nan")
    for put in ({3: inf}, {k - 1: -inf}, {70: inf}, {3: inf, 4: inf}, {3: inf, k - 2: -inf}, {3: inf, 130: nan}):
        X, row = c.X.clone(), m - 1
        for j, v in put.items():
            X[row, j] = v
        ids[row] = -1                                 # the frozen product alone
        Y = B.qlora_linear_fwd_multi(X.to(DEV), w, A, Bm, s, ids.to(DEV))
        with np.errstate(invalid="ignore"):
            _same_kind(Y[row:], R.bf16_to_f64(X[row:]) @ W.T)
        got, ref = R.bf16_to_f64(Y[:row]), R.bf16_to_f64(clean[:row])
        if m > 4 or k <= 256:
            assert np.array_equal(got, ref)
        else:
            # Up to four rows the warps' sums (256 columns each) are added in the
            # order they come: k fp32 additions on either side, and the one
            # step of bf16 (2^-7 at most) that this may move the rounding by.
            assert np.all(np.abs(got - ref) <= 2.0 ** -7 * np.abs(ref) + 2 * k * M.E * (np.abs(c.Xf[:row]) @ np.abs(W).T))
        # With an adapter T is infinite too; the one-adapter call agrees.
        ids[row] = 1
        Y = B.qlora_linear_fwd_multi(X.to(DEV), w, A, Bm, s, ids.to(DEV))
        one = B.qlora_linear_fwd(X.to(DEV), w, A[1], Bm[1], r, float(c.scale[1]))
        _same_kind(Y[row:], R.bf16_to_f64(one[row:]))
    assert B.qlora_poll_device_error() == 0
