"""GPU parity of the many-adapter layer with ``oracle/multi.py``, element by
element under the derived bounds of ``multi_refs``: every dispatch size (the
two weight-streaming kernels, one 128-row tile, CTA pairs), ranks of one to
four 64-column units and of 16- and 32-column ones, rows in runs and in any
order, adapters without rows, rows without an adapter."""
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
ORDERS = ["one", "segments", "mixed", "none", "last"]


def _fwd(c):
    A, Bm, s, ids = c.on(DEV)
    return B.qlora_linear_fwd_multi(c.X.to(DEV), c.weight(DEV), A, Bm, s, ids)


def _bwd(c, X=None, T=None, want_dx=True):
    A, Bm, s, ids = c.on(DEV)
    return B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV) if X is None else X, c.weight(DEV), A, Bm, s, ids, T=T,
                                    want_dx=want_dx)


def _T(c):
    return WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float())


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("m", [1, 4, 5, 16])
def test_forward_decode(m, order):
    c = M.case(m, 264, 1088, 32, 5, order, 1000 + m)
    c.check_fwd(_fwd(c))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("m", [17, 128, 129, 513, 1100])
def test_forward_tiles(m, order):
    c = M.case(m, 520, 192, 16, 7, order, 2000 + m)
    c.check_fwd(_fwd(c))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("r", [16, 32, 48, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("m", [3, 9, 100, 600])
def test_forward_ranks(m, r):
    c = M.case(m, 72, 320, r, 6, "mixed", 3000 + m + r)
    c.check_fwd(_fwd(c))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("m,count", [(128, 200), (600, 300), (16, 40), (40, 1)])
def test_forward_many_adapters(m, count):
    c = M.case(m, 264, 128, 16, count, "mixed", 4000 + m)
    c.check_fwd(_fwd(c))


@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("m", [1, 17, 65, 128, 300, 1100])
def test_backward(m, order):
    c = M.case(m, 264, 192, 16, 5, order, 5000 + m)
    T = _T(c)
    c.check_bwd(_bwd(c, T=T.to(DEV)), c.Xf, R.bf16_to_f64(T))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("r", [16, 32, 48, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("m", [33, 600])
def test_backward_ranks(m, r):
    c = M.case(m, 520, 128, r, 4, "mixed", 6000 + m + r)
    T = _T(c)
    c.check_bwd(_bwd(c, T=T.to(DEV)), c.Xf, R.bf16_to_f64(T))


@pytest.mark.parametrize("r", [16, 80])
@pytest.mark.parametrize("order", ["segments", "mixed"])
def test_backward_from_a_checkpoint(order, r):
    """The 8-bit checkpoint and many adapters together."""
    c = M.case(700, 72, 1088, r, 6, order, 7000 + r)
    act = B.qlora_act_quantize(c.X.to(DEV))
    T = _T(c)
    codes, scale = act8.quantize(c.Xf)
    c.check_bwd(_bwd(c, X=act, T=T.to(DEV)), act8.dequant_values(codes, scale), R.bf16_to_f64(T))


@pytest.mark.parametrize("m,count", [(128, 200), (600, 300)])
def test_backward_many_adapters(m, count):
    c = M.case(m, 72, 64, 16, count, "mixed", 8000 + m)
    T = _T(c)
    c.check_bwd(_bwd(c, T=T.to(DEV)), c.Xf, R.bf16_to_f64(T))


@pytest.mark.parametrize("m", [2, 300])
def test_adapter_terms_alone(m):
    """With a zero weight only the adapters' terms are left: a wrong adapter,
    scale or mask cannot hide behind the frozen product."""
    c = M.case(m, 264, 256, 16, 9, "mixed", 9000 + m, zero_weight=True)
    c.check_fwd(_fwd(c))
    T = _T(c)
    c.check_bwd(_bwd(c, T=T.to(DEV)), c.Xf, R.bf16_to_f64(T))


def test_training_step_takes_T_from_the_forward():
    """Forward, checkpoint, backward as a step runs them; T is the start of
    the forward's workspace; T computed by the backward gives the same dB."""
    m, n, k, r, count = 513, 264, 192, 32, 5
    c = M.case(m, n, k, r, count, "segments", 9100)
    A, Bm, s, ids = c.on(DEV)
    w, X, dY = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV)
    ws = torch.empty(B.qlora_multi_workspace_bytes(B.QLORA_OP_FWD, m, n, k, r, count), dtype=torch.uint8, device=DEV)
    Y = B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, ws=ws)
    T = ws[:m * r * 2].view(torch.bfloat16).view(m, r)
    act = B.qlora_act_quantize(X)
    got = B.qlora_linear_bwd_multi(dY, act, w, A, Bm, s, ids, T=T)
    plain = B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids)
    torch.cuda.synchronize()
    c.check_fwd(Y)
    codes, scale = act8.quantize(c.Xf)
    c.check_bwd(got, act8.dequant_values(codes, scale), R.bf16_to_f64(T))
    assert torch.equal(plain[0], got[0]) and torch.equal(plain[2], got[2])


@pytest.mark.parametrize("m", [3, 16, 100, 600])
def test_another_tenants_values_do_not_leak(m):
    """NaN and Inf in one tenant's rows and adapter reach that tenant only."""
    c = M.case(m, 72, 192, 16, 4, "mixed", 9200 + m)
    base = _fwd(c)
    gA, gB = _bwd(c, T=_T(c).to(DEV))[1:]
    torch.cuda.synchronize()
    sick = 2
    rows = torch.from_numpy(np.nonzero(c.ids_np == sick)[0])
    others = torch.from_numpy(np.nonzero(c.ids_np != sick)[0]).to(DEV)
    T = _T(c)
    c.X[rows] = float("nan")
    c.dY[rows] = float("inf")
    T[rows] = float("nan")
    c.A[sick] = float("inf")
    c.B[sick] = float("nan")
    Y = _fwd(c)
    dX, dA, dB = _bwd(c, T=T.to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(Y[others], base[others])
    rest = [a for a in range(4) if a != sick]
    assert torch.equal(dA[rest], gA[rest]) and torch.equal(dB[rest], gB[rest])
    assert bool(torch.isfinite(dX[others].float()).all())


def test_results_do_not_depend_on_the_run():
    c = M.case(1100, 264, 1088, 48, 11, "mixed", 9300)
    T = _T(c).to(DEV)
    Y0, g0 = _fwd(c), _bwd(c, T=T)
    for _ in range(3):
        assert torch.equal(_fwd(c), Y0)
        for a, b in zip(_bwd(c, T=T), g0):
            assert torch.equal(a, b)


def test_captured_call_follows_new_ids():
    """ids are read on the device: a replay after an update uses the new
    ones; two graphs on their own workspaces replay on two streams."""
    m, n, k, r, count = 200, 264, 192, 16, 6
    c1, c2 = (M.case(m, n, k, r, count, o, 9400) for o in ("segments", "mixed"))
    w, X = c1.weight(DEV), c1.X.to(DEV)
    A, Bm, s, _ = c1.on(DEV)
    ids = c1.ids.to(DEV)
    nbytes = B.qlora_multi_workspace_bytes(B.QLORA_OP_FWD, m, n, k, r, count)
    graphs = []
    for _ in range(2):
        out = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
        B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, out=out, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, out=out, ws=ws)
        graphs.append((g, out, ws))
    want1 = B.qlora_linear_fwd_multi(X, w, A, Bm, s, c1.ids.to(DEV))
    want2 = B.qlora_linear_fwd_multi(X, w, A, Bm, s, c2.ids.to(DEV))
    for want, src in ((want1, c1.ids), (want2, c2.ids)):
        ids.copy_(src)
        torch.cuda.synchronize()
        for g, out, _ in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        for _, out, _ in graphs:
            assert torch.equal(out, want)


def test_backward_without_input_gradient_and_empty_batch():
    c = M.case(150, 72, 128, 16, 3, "segments", 9500)
    T = _T(c)
    dX, dA, dB = _bwd(c, T=T.to(DEV), want_dx=False)
    assert dX is None
    c.check_bwd((None, dA, dB), c.Xf, R.bf16_to_f64(T))
    A, Bm, s, ids = c.on(DEV)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    dX, dA, dB = B.qlora_linear_bwd_multi(torch.empty(0, 72, dtype=torch.bfloat16, device=DEV), e, c.weight(DEV), A, Bm, s,
                                          ids[:0])
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()
    assert B.qlora_linear_fwd_multi(e, c.weight(DEV), A, Bm, s, ids[:0]).shape == (0, 72)


def test_slices_of_ids_and_scale_need_no_wider_alignment():
    c = M.case(60, 72, 128, 16, 4, "mixed", 9600)
    A, Bm, s, ids = c.on(DEV)
    pad_i = torch.cat([ids[:1], ids])[1:]
    pad_s = torch.cat([s[:1], s])[1:]
    Y = B.qlora_linear_fwd_multi(c.X.to(DEV), c.weight(DEV), A, Bm, pad_s, pad_i)
    assert torch.equal(Y, _fwd(c))


def test_other_weight_formats():
    """FP4 codes and the E4M3 + mean absmax format go through the same kernels."""
    for m in (2, 12, 90, 300):
        c = M.case(m, 72, 256, 16, 3, "mixed", 9700 + m)
        A, Bm, s, ids = c.on(DEV)
        for cb, fmt in ((B.QLORA_CODEBOOK_FP4, B.QLORA_DQ_LINEAR8), (B.QLORA_CODEBOOK_NF4, B.QLORA_DQ_FP8_MEAN)):
            w = B.qlora_quantize_4bit_dq(c.W.to(DEV), cb, dq_format=fmt)
            Y = B.qlora_linear_fwd_multi(c.X.to(DEV), w, A, Bm, s, ids)
            W = B.qlora_dequant(w).double().cpu().numpy()
            ref = M.multi.fwd(c.Xf, W, c.Af, c.Bf, c.s, c.ids_np)
            assert R.err(R.bf16_to_f64(Y), ref) <= 2e-2


def test_refusals_on_the_gpu():
    c = M.case(20, 72, 128, 16, 3, "mixed", 9800)
    A, Bm, s, ids = c.on(DEV)
    w, X, dY = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV)
    bad = [dict(ids=ids.long()), dict(ids=ids[:-1]), dict(s=s.double()), dict(s=s[:2]), dict(Bm=Bm[:2]),
           dict(A=A.float()), dict(X=X[:, :64]), dict(X=X.t().contiguous().t()), dict(ids=ids.cpu())]
    for kw in bad:
        a = dict(X=X, A=A, Bm=Bm, s=s, ids=ids)
        a.update(kw)
        with pytest.raises(ValueError):
            B.qlora_linear_fwd_multi(a["X"], w, a["A"], a["Bm"], a["s"], a["ids"])
    with pytest.raises(B.QLoRAError):
        B.qlora_linear_bwd_multi(dY, B.qlora_act_quantize(X), w, A, Bm, s, ids)          # a checkpoint without T
    with pytest.raises(ValueError):
        B.qlora_linear_bwd_multi(dY, B.qlora_act_quantize(X[:10]), w, A, Bm, s, ids, T=_T(c).to(DEV))
    with pytest.raises(B.QLoRAError):
        B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
