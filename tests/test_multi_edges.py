"""Calls of the many-adapter layer that its documentation allows and that lie
off the beaten track: exact workspaces, two streams at once, two graphs on one
workspace, a first call inside a capture, padded rows full of NaN, the largest
sets, batches of many tiles, checkpoints of non-finite values."""
import os
import subprocess
import sys

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
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _T(c):
    return WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float())


def _guarded(size):
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    return ws[:size], ws[size:]


@pytest.mark.parametrize("r", [16, 48, 256])
@pytest.mark.parametrize("m,count", [(1, 1), (17, 40), (65, 1), (130, 9), (513, 70)])
def test_workspace_of_exactly_the_stated_size(m, count, r):
    n, k = 72, 192
    c = M.case(m, n, k, r, count, "mixed", 11000 + m + r)
    A, Bm, s, ids = c.on(DEV)
    ws, guard = _guarded(B.qlora_multi_workspace_bytes(B.QLORA_OP_FWD, m, n, k, r, count))
    Y = B.qlora_linear_fwd_multi(c.X.to(DEV), c.weight(DEV), A, Bm, s, ids, ws=ws)
    ws2, guard2 = _guarded(B.qlora_multi_workspace_bytes(B.QLORA_OP_LORA_BWD, m, n, k, r, count))
    T = _T(c)
    got = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), c.weight(DEV), A, Bm, s, ids, T=T.to(DEV), ws=ws2)
    torch.cuda.synchronize()
    assert bool((guard == 0xA5).all()) and bool((guard2 == 0xA5).all())
    c.check_fwd(Y)
    c.check_bwd(got, c.Xf, R.bf16_to_f64(T))


def test_two_streams_at_once():
    """Calls of different shapes on two streams, again and again, give what
    each gives alone."""
    cases = [M.case(700, 264, 1088, 32, 6, "mixed", 11100), M.case(150, 520, 192, 16, 9, "segments", 11101)]
    calls = []
    for c in cases:
        A, Bm, s, ids = c.on(DEV)
        w, X, dY, T = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV), _T(c).to(DEV)
        size = max(B.qlora_multi_workspace_bytes(op, *dY.shape, X.shape[1], A.shape[1], A.shape[0])
                   for op in (B.QLORA_OP_FWD, B.QLORA_OP_LORA_BWD))
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        calls.append(lambda w=w, X=X, dY=dY, T=T, A=A, Bm=Bm, s=s, ids=ids, ws=ws:
                     (B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, ws=ws),
                      *B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids, T=T, ws=ws)))
    alone = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = []
        for st, f in zip(streams, calls):
            with torch.cuda.stream(st):
                got.append(f())
        torch.cuda.synchronize()
        for g, a in zip(got, alone):
            assert all(torch.equal(x, y) for x, y in zip(g, a))
    assert B.qlora_poll_device_error() == 0


def test_two_graphs_share_a_workspace():
    c, d = M.case(300, 264, 192, 16, 5, "mixed", 11200), M.case(90, 264, 192, 16, 5, "segments", 11201)
    w = c.weight(DEV)
    ws = torch.empty(B.qlora_multi_workspace_bytes(B.QLORA_OP_FWD, 300, 264, 192, 16, 5), dtype=torch.uint8, device=DEV)
    graphs, outs, refs = [], [], []
    for x in (c, d):
        A, Bm, s, ids = x.on(DEV)
        X = x.X.to(DEV)
        out = torch.empty(X.shape[0], 264, dtype=torch.bfloat16, device=DEV)
        refs.append(B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids).clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, out=out, ws=ws)
        graphs.append((g, A, Bm, s, ids, X))
        outs.append(out)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], refs[i])


FIRST_CALL = """
import sys, torch
sys.path[:0] = [{root!r}, {tests!r}]
import multi_refs as M
from bit_nf4_quantized_qlora_b200 import binding as B
dev = "cuda:0"
c = M.case(200, 264, 192, 32, 5, "mixed", 11300)
A, Bm, s, ids = c.on(dev)
w, X, dY = c.weight(dev), c.X.to(dev), c.dY.to(dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    Y = B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids)
    act = B.qlora_act_quantize(X)
    got = B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids)
g.replay()
torch.cuda.synchronize()
c.check_fwd(Y)
again = B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids)
assert all(torch.equal(a, b) for a, b in zip(got, again))
assert torch.equal(act.codes, B.qlora_act_quantize(X).codes)
assert B.qlora_poll_device_error() == 0
print("first call captured")
"""


def test_the_first_call_of_a_process_may_be_captured():
    code = FIRST_CALL.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "first call captured" in run.stdout, run.stderr[-2000:]


@pytest.mark.parametrize("m", [12, 200, 700])
def test_padded_rows_of_nan_reach_nobody(m):
    """Rows without an adapter behind the last sequence, NaN in X and dY: the
    others' Y and dX, and every gradient, are as without them."""
    pad = 37
    c = M.case(m, 264, 192, 16, 4, "segments", 11400 + m)
    A, Bm, s, ids = c.on(DEV)
    w, X, dY, T = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV), _T(c).to(DEV)
    nan = lambda t: torch.cat([t, torch.full((pad, t.shape[1]), float("nan"), dtype=t.dtype, device=DEV)])
    ids_p = torch.cat([ids, torch.full((pad,), -1, dtype=torch.int32, device=DEV)])
    Y = B.qlora_linear_fwd_multi(nan(X), w, A, Bm, s, ids_p)
    dX, dA, dB = B.qlora_linear_bwd_multi(nan(dY), nan(X), w, A, Bm, s, ids_p, T=nan(T))
    torch.cuda.synchronize()
    if m > 16:       # the padded batch takes the same kernels
        c.check_fwd(Y[:m])
    c.check_bwd((dX[:m], dA, dB), c.Xf, R.bf16_to_f64(T))
    assert bool(Y[m:].isnan().all()) and bool(dX[m:].isnan().all())


def test_the_largest_set_of_adapters():
    """65535 adapters, of which a few have rows: each row's result and each
    present adapter's gradients are those of a small set."""
    m, n, k, r, few = 300, 72, 64, 16, 7
    c = M.case(m, n, k, r, few, "mixed", 11500)
    count = 65535
    where = torch.tensor([0, 1, 4095, 30000, 30001, 65533, 65534])
    A = torch.zeros(count, r, k, dtype=torch.bfloat16, device=DEV)
    Bm = torch.zeros(count, n, r, dtype=torch.bfloat16, device=DEV)
    s = torch.ones(count, device=DEV)
    A[where], Bm[where], s[where] = c.A.to(DEV), c.B.to(DEV), c.scale.to(DEV)
    inside = (c.ids >= 0) & (c.ids < few)
    ids = torch.where(inside, where[c.ids.clamp(0, few - 1).long()].int(), torch.full_like(c.ids, -1)).to(DEV)
    w = c.weight(DEV)
    c.check_fwd(B.qlora_linear_fwd_multi(c.X.to(DEV), w, A, Bm, s, ids))
    T = _T(c)
    dX, dA, dB = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), w, A, Bm, s, ids, T=T.to(DEV))
    c.check_bwd((dX, dA[where].contiguous(), dB[where].contiguous()), c.Xf, R.bf16_to_f64(T))
    dA[where], dB[where] = 0, 0
    assert not dA.any() and not dB.any()
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("order", ["segments", "mixed"])
def test_batches_of_many_tiles(order):
    """More 64-row slots than clusters of any size."""
    m, n, k, r, count = 40001, 72, 64, 16, 11
    c = M.case(m, n, k, r, count, order, 11600)
    A, Bm, s, ids = c.on(DEV)
    c.check_fwd(B.qlora_linear_fwd_multi(c.X.to(DEV), c.weight(DEV), A, Bm, s, ids))
    T = _T(c)
    got = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), c.weight(DEV), A, Bm, s, ids, T=T.to(DEV))
    c.check_bwd(got, c.Xf, R.bf16_to_f64(T))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.parametrize("r", [16, 64, 80])
@pytest.mark.parametrize("few", [1, 64, 65, 177, 300])
@pytest.mark.parametrize("count", [1, 3])
def test_few_rows_with_an_adapter_among_many_without(few, count, r):
    """Fewer 64-row slots than the batch has room for: gradients of a group
    that crosses CTAs, some of which have no slot."""
    m, n, k = 1200, 264, 192
    c = M.case(m, n, k, r, count, "none", 11700 + few + r)
    g = np.random.default_rng(few)
    ids = np.full(m, -1, dtype=np.int32)
    ids[g.choice(m, few, replace=False)] = count - 1
    c = M.Case(c.W, c.X, c.dY, c.A, c.B, c.scale, torch.from_numpy(ids))
    A, Bm, s, idd = c.on(DEV)
    c.check_fwd(B.qlora_linear_fwd_multi(c.X.to(DEV), c.weight(DEV), A, Bm, s, idd))
    T = _T(c)
    for X, Xf in ((c.X.to(DEV), c.Xf), (B.qlora_act_quantize(c.X.to(DEV)), act8.dequant_values(*act8.quantize(c.Xf)))):
        got = B.qlora_linear_bwd_multi(c.dY.to(DEV), X, c.weight(DEV), A, Bm, s, idd, T=T.to(DEV))
        c.check_bwd(got, Xf, R.bf16_to_f64(T))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_non_finite_value_stays_visible_in_its_block(bad):
    X = WL.bf16(WL.normal((3, 192), 1.0, 8)).to(DEV)
    ref = B.qlora_act_dequant(B.qlora_act_quantize(X))
    sick = X.clone()
    sick[1, 70] = bad
    got = B.qlora_act_dequant(B.qlora_act_quantize(sick))
    torch.cuda.synchronize()
    assert not got[1, 64:128].isfinite().any()
    got[1, 64:128] = ref[1, 64:128]
    assert torch.equal(got, ref)
