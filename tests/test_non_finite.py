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
