"""Many adapters past 32-bit element counts, adapters that are loaded and have
no rows, and backwards that form the adapter gradients alone."""
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
PERIOD = 512                                       # rows of the tallest tile


def _small_integers(shape, values, seed):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.choice(np.asarray(values, dtype=np.float32), size=shape)).to(torch.bfloat16)


@pytest.mark.parametrize("n,k", [(1024, 64), (64, 1024)])
def test_the_longest_batch(n, k):
    """2^22 rows, so that X or Y, dY or dX hold 2^32 elements.  Rows repeat every
    512, a tile: every tile's Y and dX are the first one's.  The gradients' terms are
    small integers times powers of two, exact in fp32, so that they are the
    period's sums times the number of periods, rounded once."""
    m, r, count, tiles = 1 << 22, 16, 5, (1 << 22) // PERIOD
    c = M.case(PERIOD, n, k, r, count, "mixed", 17000 + n)
    w = c.weight(DEV)
    A = _small_integers((count, r, k), (-1, 0, 1), 1).to(DEV) / 64
    Bm = _small_integers((count, n, r), (-1, 0, 0, 1), 2).to(DEV) / 16
    s = torch.tensor([0.25, 0.5, 1.0, 2.0, 1.0], device=DEV)
    X1, dY1 = _small_integers((PERIOD, k), (-1, 0, 1), 3).to(DEV), _small_integers((PERIOD, n), (-1, 0, 0, 0, 1), 4).to(DEV)
    T1 = _small_integers((PERIOD, r), (-1, 0, 1), 5).to(DEV)
    ids1 = c.ids.to(DEV)
    X, dY, T, ids = (t.repeat(tiles, *([1] * (t.dim() - 1))) for t in (X1, dY1, T1, ids1))
    p = M.Case(c.W, X1.cpu(), dY1.cpu(), A.cpu(), Bm.cpu(), s.cpu(), c.ids)
    Y = B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids)
    Yt = Y.view(tiles, PERIOD, n)
    assert torch.equal(Yt, Yt[:1].expand_as(Yt))
    p.check_fwd(Yt[0])
    del Y, Yt
    dX, dA, dB = B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids, T=T)
    dXt = dX.view(tiles, PERIOD, k)
    assert torch.equal(dXt, dXt[:1].expand_as(dXt))
    p.check_bwd((dXt[0], *B.qlora_linear_bwd_multi(dY1, X1, w, A, Bm, s, ids1, T=T1)[1:]), p.Xf, R.bf16_to_f64(T1))
    live = ((ids1 >= 0) & (ids1 < count))
    U = torch.zeros(PERIOD, r, dtype=torch.float64, device=DEV)
    wA, wB = torch.zeros(A.shape, dtype=torch.float64, device=DEV), torch.zeros(Bm.shape, dtype=torch.float64, device=DEV)
    for a in range(count):
        i = live & (ids1 == a)
        U[i] = s[a].double() * (dY1[i].double() @ Bm[a].double())
        assert torch.equal(U[i].to(torch.bfloat16).double(), U[i])          # so U's rounding changes nothing
        wA[a], wB[a] = U[i].t() @ X1[i].double(), dY1[i].double().t() @ T1[i].double()
        # Every partial sum is a whole number below 2^24 of the terms' unit, s_a / 16.
        assert float((U[i].abs().t() @ X1[i].double().abs()).max()) * tiles * 16 / float(s[a]) < 2 ** 24
    assert torch.equal(dA, (wA * tiles).to(torch.bfloat16)) and torch.equal(dB, (wB * tiles).to(torch.bfloat16))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("m", [3, 12, 100, 300])
def test_sets_past_32_bits(m):
    """65535 adapters of a 4096-column projection: B and dB hold 2^32 elements."""
    n, k, r, few, count = 4096, 64, 16, 4, 65535
    c = M.case(m, n, k, r, few, "mixed", 17100 + m)
    where = torch.tensor([0, 32768, 65533, 65534])
    A = torch.zeros(count, r, k, dtype=torch.bfloat16, device=DEV)
    Bm = torch.zeros(count, n, r, dtype=torch.bfloat16, device=DEV)
    s = torch.ones(count, device=DEV)
    A[where], Bm[where], s[where] = c.A.to(DEV), c.B.to(DEV), c.scale.to(DEV)
    inside = (c.ids >= 0) & (c.ids < few)
    ids = torch.where(inside, where[c.ids.clamp(0, few - 1).long()].int(), torch.full_like(c.ids, -1)).to(DEV)
    w = c.weight(DEV)
    c.check_fwd(B.qlora_linear_fwd_multi(c.X.to(DEV), w, A, Bm, s, ids))
    T = WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float())
    dX, dA, dB = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), w, A, Bm, s, ids, T=T.to(DEV))
    c.check_bwd((dX, dA[where].contiguous(), dB[where].contiguous()), c.Xf, R.bf16_to_f64(T))
    dA[where], dB[where] = 0, 0
    assert not dA.any() and not dB.any()
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("m", [1, 4, 16, 60, 300])
def test_absent_adapters_values_reach_nobody(m):
    """Loaded adapters without rows, NaN throughout."""
    c = M.case(m, 264, 192, 32, 6, "mixed", 17200 + m)
    ids = torch.where((c.ids >= 0) & (c.ids < 6), c.ids % 3 * 2, c.ids)          # 0, 2 and 4
    c.A[1::2], c.B[1::2], c.scale[1::2] = float("nan"), float("nan"), float("nan")
    clean = M.Case(c.W, c.X, c.dY, torch.nan_to_num(c.A), torch.nan_to_num(c.B), torch.nan_to_num(c.scale), ids)
    A, Bm, s = (t.to(DEV) for t in (c.A, c.B, c.scale))
    w, idd = clean.weight(DEV), ids.to(DEV)
    clean.check_fwd(B.qlora_linear_fwd_multi(c.X.to(DEV), w, A, Bm, s, idd))
    T = WL.bf16(torch.from_numpy(M.multi.lora_t(clean.Xf, clean.Af, clean.s, clean.ids_np)).float())
    got = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), w, A, Bm, s, idd, T=T.to(DEV))
    clean.check_bwd(got, clean.Xf, R.bf16_to_f64(T))


@pytest.mark.parametrize("r", [16, 128])
@pytest.mark.parametrize("m", [50, 300])
def test_gradients_of_a_checkpoint_without_the_inputs(m, r):
    c = M.case(m, 264, 320, r, 1, "one", 17300 + m + r)
    w, dY, act = c.weight(DEV), c.dY.to(DEV), B.qlora_act_quantize(c.X.to(DEV))
    A, Bm, s, ids = c.on(DEV)
    T = WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float())
    Xh = act8.dequant_values(*act8.quantize(c.Xf))
    one = B.qlora_linear_bwd_act8(dY, act, w, A[0], Bm[0], r, float(c.s[0]), T.to(DEV), want_dx=False)
    many = B.qlora_linear_bwd_multi(dY, act, w, A, Bm, s, ids, T=T.to(DEV), want_dx=False)
    assert one[0] is None and many[0] is None
    c.check_bwd((None, one[1][None], one[2][None]), Xh, R.bf16_to_f64(T))
    c.check_bwd(many, Xh, R.bf16_to_f64(T))
