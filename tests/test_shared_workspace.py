"""One workspace for the forward and the backward: T, which the forward leaves
at the start of its workspace, may lie in the backward's; the backward then
keeps U off it.  A T anywhere else in a workspace, where the backward writes,
is refused."""
import ctypes

import pytest
import torch

import multi_refs as M
import oracle_refs as R
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import workloads as WL
from oracle import act8

DEV = "cuda:0"
P = 0x10000000
WS = 0x20000000
M_, N_, K_, R_ = 40, 1024, 1024, 16
MR = 1280                                          # m r bf16 values, a multiple of 256 bytes


def _call(name, T, ws_bytes=1 << 22):
    """The entry point with T at address `T` and its workspace at WS."""
    lib = B.lib()
    w = B.NF4WeightC(P, P, P, N_, K_, 64, 256)
    act = B.Act8C(P, P, M_, K_)
    if name == "bwd":
        return lib.qlora_linear_bwd(P, P, T, M_, ctypes.byref(w), P, P, R_, 1.0, P, P, P, WS, ws_bytes, None)
    if name == "bwd_act8":
        return lib.qlora_linear_bwd_act8(P, ctypes.byref(act), T, M_, ctypes.byref(w), P, P, R_, 1.0, P, P, P, WS,
                                         ws_bytes, None)
    s = B.AdapterSetC(P, P, P, 4, R_)
    return lib.qlora_linear_bwd_multi(P, P, None, T, M_, ctypes.byref(w), ctypes.byref(s), P, P, P, P, WS, ws_bytes, None)


@pytest.mark.parametrize("name", ["bwd", "bwd_act8", "bwd_multi"])
def test_a_T_where_the_backward_writes_is_refused(name):
    need = (B.qlora_multi_workspace_bytes(B.QLORA_OP_LORA_BWD, M_, N_, K_, R_, 4) if name == "bwd_multi"
            else B.qlora_workspace_bytes(B.QLORA_OP_LORA_BWD, M_, N_, K_, R_))
    assert need > 2 * MR
    # Across the start of the workspace, across its first two parts, into what follows them.
    for T in (WS - 16, WS - MR + 16, WS + 16, WS + MR - 16, WS + MR + 16, WS + 2 * MR, WS + need - 16):
        assert _call(name, T) == B.QLORA_ERR_WORKSPACE, hex(T)


ORDERS = [(20, "mixed"), (130, "segments"), (600, "mixed")]


def _T_of(c):
    return WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float()).to(DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("m,order", ORDERS)
def test_forward_and_backward_in_one_workspace(m, order, keep8):
    n, k, r, count = 264, 192, 16, 5
    c = M.case(m, n, k, r, count, order, 13000 + m)
    A, Bm, s, ids = c.on(DEV)
    w, X, dY = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV)
    size = max(B.qlora_multi_workspace_bytes(op, m, n, k, r, count) for op in (B.QLORA_OP_FWD, B.QLORA_OP_LORA_BWD))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, ws=ws)
    T = ws[:m * r * 2].view(torch.bfloat16).view(m, r)
    kept = T.clone()
    src = B.qlora_act_quantize(X) if keep8 else X
    got = B.qlora_linear_bwd_multi(dY, src, w, A, Bm, s, ids, T=T, ws=ws)
    assert torch.equal(T, kept)
    want = B.qlora_linear_bwd_multi(dY, src, w, A, Bm, s, ids, T=kept)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    Xf = act8.dequant_values(*act8.quantize(c.Xf)) if keep8 else c.Xf
    c.check_bwd(got, Xf, R.bf16_to_f64(kept))


@pytest.mark.gpu
@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("m,r", [(1, 16), (77, 48), (300, 16), (300, 128)])
def test_one_adapter_forward_and_backward_in_one_workspace(m, r, keep8, at):
    """T in the first part of the workspace, where the forward leaves it, or the second."""
    n, k = 264, 192
    c = M.case(m, n, k, r, 1, "one", 13100 + m + r)
    s = float(c.s[0])
    w, X, dY, A, Bm = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV), c.A[0].to(DEV), c.B[0].to(DEV)
    ws = torch.empty(B.qlora_workspace_bytes(B.QLORA_OP_LORA_BWD, m, n, k, r), dtype=torch.uint8, device=DEV)
    B.qlora_linear_fwd(X, w, A, Bm, r, s, ws=ws)
    lo = at * (-(-m * r * 2 // 256) * 256)
    T = ws[lo:lo + m * r * 2].view(torch.bfloat16).view(m, r)
    kept = ws[:m * r * 2].view(torch.bfloat16).view(m, r).clone()
    T.copy_(kept)
    if keep8:
        act = B.qlora_act_quantize(X)
        run = lambda T, ws: B.qlora_linear_bwd_act8(dY, act, w, A, Bm, r, s, T, ws=ws)
    else:
        run = lambda T, ws: B.qlora_linear_bwd(dY, X, w, A, Bm, r, s, T=T, ws=ws)
    got, want = run(T, ws), run(kept, None)
    assert torch.equal(T, kept) and all(torch.equal(a, b) for a, b in zip(got, want))
    Xf = act8.dequant_values(*act8.quantize(c.Xf)) if keep8 else c.Xf
    c.check_bwd((got[0], got[1][None], got[2][None]), Xf, R.bf16_to_f64(kept))
