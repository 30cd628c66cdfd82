"""The autograd modules of many adapters (``MultiQLoRALinear``) and of 8-bit
input checkpoints (``act8``), alone and in the decoder block, against
``oracle/multi.py`` and ``oracle/act8.py`` under the element-wise bounds of
``multi_refs``, and against differences of the loss."""
import copy

import numpy as np
import pytest
import torch

import multi_refs as M
import oracle_refs as R
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import layer as L
from bit_nf4_quantized_qlora_b200 import workloads as WL
from oracle import act8

DEV = "cuda:0"


def _module(c, **kw):
    return L.MultiQLoRALinear(c.weight(DEV), c.A.to(DEV), c.B.to(DEV), c.scale.to(DEV), **kw)


def _restored(X):
    return act8.dequant_values(*act8.quantize(R.bf16_to_f64(X)))


def _lora_T(c):
    return R.bf16_to_f64(WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float()))


def test_adapters_of_lower_rank_are_padded_with_zeros():
    A0, A1 = torch.ones(8, 64), torch.ones(40, 64)
    m = L.MultiQLoRALinear.from_adapters(B.NF4Weight(None, None, None, 24, 64),
                                         [(A0, torch.ones(24, 8), 16.0), (A1, torch.ones(24, 40), 10.0)])
    assert m.A.shape == (2, 48, 64) and m.B.shape == (2, 24, 48) and m.scale.tolist() == [2.0, 0.25]
    assert m.A[0].sum() == 8 * 64 and m.A[1].sum() == 40 * 64 and not m.A[0, 8:].any() and not m.B[1, :, 40:].any()


def test_ids_and_checkpoints_must_fit_the_input():
    m = L.MultiQLoRALinear(B.NF4Weight(None, None, None, 24, 64), torch.zeros(2, 16, 64), torch.zeros(2, 24, 16),
                           torch.ones(2))
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    for shape in ((3,), (2, 4), (2, 3, 1)):
        with pytest.raises(ValueError):
            m(x, torch.zeros(shape, dtype=torch.int32))
    act = B.Act8(torch.zeros(5, 64, dtype=torch.int8), torch.zeros(5, 1, dtype=torch.bfloat16), 5, 64)
    with pytest.raises(ValueError):
        m(x, torch.zeros(2, dtype=torch.int32), act=act)
    lin = L.QLoRALinear(B.NF4Weight(None, None, None, 24, 64), torch.zeros(16, 64), torch.zeros(24, 16), 1.0)
    with pytest.raises(ValueError):
        lin(x, act=act)


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("m,order", [(1, "last"), (12, "mixed"), (96, "segments"), (600, "mixed"), (600, "none")])
def test_module_and_its_gradients(m, order, keep8):
    c = M.case(m, 264, 192, 16, 5, order, 300 + m)
    lin = _module(c, act8=keep8)
    X = c.X.to(DEV).requires_grad_(True)
    Y = lin(X, c.ids.to(DEV))
    Y.backward(c.dY.to(DEV))
    c.check_fwd(Y)
    with torch.no_grad():
        assert torch.equal(lin(X, c.ids.to(DEV)), Y)
    # The module's T is its forward's, itself within one rounding and the
    # accumulation of the formula's, which the bound on dB adds.
    T = B.qlora_multi_workspace_bytes(B.QLORA_OP_FWD, m, 264, 192, 16, 5)
    ws = torch.empty(T, dtype=torch.uint8, device=DEV)
    B.qlora_linear_fwd_multi(c.X.to(DEV), lin.w, lin.A.detach(), lin.B.detach(), lin.scale, c.ids.to(DEV), ws=ws)
    T = R.bf16_to_f64(ws[:m * 32].view(torch.bfloat16).view(m, 16))
    ref = M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)
    Ta = M.multi.lora_t(np.abs(c.Xf), np.abs(c.Af), c.s, c.ids_np)
    assert np.all(np.abs(T - ref) <= M.H * np.abs(ref) + 2 * 192 * M.E * Ta)
    c.check_bwd((X.grad, lin.A.grad, lin.B.grad), _restored(c.X) if keep8 else c.Xf, T)
    assert B.qlora_poll_device_error() == 0


@pytest.mark.gpu
def test_one_id_per_sequence_is_one_per_row():
    c = M.case(40, 264, 192, 16, 5, "mixed", 350)
    lin = _module(c)
    x = c.X.to(DEV).view(4, 10, 192)
    seq = torch.tensor([3, -1, 0, 3], dtype=torch.int32, device=DEV)
    with torch.no_grad():
        y = lin(x, seq)
        assert torch.equal(y, lin(x, seq[:, None].expand(4, 10)))
        assert torch.equal(y.view(40, 264), lin(c.X.to(DEV), seq.repeat_interleave(10)))
        assert lin(x[:0], seq[:0]).shape == (0, 10, 264)


@pytest.mark.gpu
def test_adapters_padded_to_one_rank_act_as_their_own():
    """Against the one-adapter layer of each rank: the same products, but the
    padded T comes from the many-adapter kernels, so within the bounds."""
    c = M.case(64, 264, 192, 32, 2, "segments", 360)
    c.A[0, 16:], c.B[0, :, 16:] = 0, 0
    c = M.Case(c.W, c.X, c.dY, c.A, c.B, torch.tensor([2.0, 0.25]), c.ids)
    lin = L.MultiQLoRALinear.from_adapters(c.weight(DEV), [(c.A[0, :16].to(DEV), c.B[0, :, :16].to(DEV), 32.0),
                                                           (c.A[1].to(DEV), c.B[1].to(DEV), 8.0)])
    X = c.X.to(DEV).requires_grad_(True)
    Y = lin(X, c.ids.to(DEV))
    Y.backward(c.dY.to(DEV))
    c.check_fwd(Y)
    assert torch.equal(lin.A, c.A.to(DEV)) and torch.equal(lin.B, c.B.to(DEV))
    assert not lin.B.grad[0, :, 16:].any() and not lin.A.grad[0, 16:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
def test_gradients_against_differences(keep8):
    """loss = sum(G Y) is linear in each of X, A and B, so L(p + D) - L(p) =
    <dL/dp, D> for any D, up to roundings.  D = a power of two times the
    gradient's sign, so that p + D and every product with D is off by known
    roundings only, and <dL/dp, D> is as large as |D| allows.

    The bound adds, in quadrature and at six times the deviation, the independent
    roundings of Y (H / sqrt 3 of each value, twice), of the two T's through B
    and of the gradient; p + D is formed and rounded first, D is what is left."""
    m, n, k, r, count = 200, 264, 192, 16, 3
    c = M.case(m, n, k, r, count, "segments", 370)
    lin = _module(c, act8=keep8)
    X = c.X.to(DEV).requires_grad_(True)
    G = c.dY.to(DEV)
    ids = c.ids.to(DEV)
    Y0 = lin(X, ids)
    gX, gA, gB = torch.autograd.grad(Y0, (X, lin.A, lin.B), G)
    Gd = G.double()

    def parts(y, x):
        """Squares of the deviations of Y's rounding and of T's through B."""
        t = torch.zeros(m, r, dtype=torch.float64, device=DEV)
        gb = torch.zeros(m, r, dtype=torch.float64, device=DEV)
        for a in range(count):
            i = ids == a
            t[i] = lin.scale[a].double() * (x[i].double() @ lin.A[a].detach().double().T)
            gb[i] = Gd[i] @ lin.B[a].detach().double()
        return ((Gd * y.double()) ** 2).sum() / 3 + ((t * gb) ** 2).sum() / 3

    for p, g, step in ((X, gX, 2.0 ** -3), (lin.A, gA, 2.0 ** -6), (lin.B, gB, 2.0 ** -5)):
        old = p.detach().clone()
        with torch.no_grad():
            var = parts(Y0.detach(), X)
            p.copy_(old + step * torch.sign(g))
            D = p.double() - old.double()
            Y1 = lin(X, ids)
            var = var + parts(Y1, X)
            p.copy_(old)
        got = (Gd * (Y1.double() - Y0.detach().double())).sum()
        want = (g.double() * D).sum()
        # The gradient's own roundings; U's or T's through the other factor is
        # of the same size as the gradient's terms.
        var = var + 2 * ((g.double() * D) ** 2).sum() / 3
        err, tol = abs(float(got - want)), 6 * M.H * float(var) ** 0.5
        if keep8 and p is lin.A:        # X^ for X: at most half a step, and its rounding, of each element
            U = torch.zeros(m, r, dtype=torch.float64, device=DEV)
            for a in range(count):
                U[ids == a] = lin.scale[a].double() * (Gd[ids == a] @ lin.B[a].detach().double())
            dX = torch.from_numpy(_restored(c.X) - c.Xf).to(DEV)
            tol += abs(float(sum(((U[ids == a].T @ dX[ids == a]) * D[a]).sum() for a in range(count))))
        assert err <= tol and tol <= 0.2 * float(want.abs()), (err, tol, float(want))


@pytest.mark.gpu
def test_one_adapter_module_with_a_checkpoint():
    """Y, dX and dB are those without the checkpoint, dA reads X^."""
    c = M.case(300, 264, 1088, 32, 1, "one", 380)
    s = float(c.scale[0])
    w = c.weight(DEV)
    lin = L.QLoRALinear(w, c.A[0].to(DEV), c.B[0].to(DEV), s * 32)
    lin8 = L.QLoRALinear(w, c.A[0].to(DEV), c.B[0].to(DEV), s * 32, act8=True)
    X, X8 = (c.X.to(DEV).requires_grad_(True) for _ in range(2))
    Y, Y8 = lin(X), lin8(X8)
    Y.backward(c.dY.to(DEV))
    Y8.backward(c.dY.to(DEV))
    assert torch.equal(Y, Y8) and torch.equal(X.grad, X8.grad) and torch.equal(lin.B.grad, lin8.B.grad)
    tol = _bound_dA(c.dYf, c.Bf[0], s, _restored(c.X))
    M.within(lin8.A.grad, *tol)
    with torch.no_grad():
        assert torch.equal(lin8(X8), Y)


def _bound_dA(dY, Bm, s, X):
    """(dA, its bound) of one adapter: see multi_refs."""
    m, n = dY.shape
    U, Ua = s * (dY @ Bm), s * (np.abs(dY) @ np.abs(Bm))
    ref = U.T @ X
    return ref, (M.H * np.abs(ref) + M.H * (1 + M.H) * (np.abs(U).T @ np.abs(X))
                 + 2 * (n + m) * M.E * (Ua.T @ np.abs(X)))


@pytest.mark.gpu
def test_decoder_block_with_checkpoints():
    """The same outputs, input gradient and B gradients bit for bit; each A
    gradient that of its projection's restored input (o keeps its own); three
    checkpoints for six projections; less memory held between forward and
    backward."""
    case = WL.DecoderLayerCase(batch=2, seq=64, hidden=256, heads=4, mlp=704, r=16, alpha=32.0)
    plain = L.build_decoder(case, torch.device(DEV))
    block = L.DecoderLayer(case.heads, {p: copy.deepcopy(plain.lin[p]) for p in L.PROJECTIONS}, act8=True)
    seen, made = {}, []
    for name, lin in block.lin.items():
        def hook(mod, args, out, name=name):
            seen[name] = [args[0].detach().reshape(-1, args[0].shape[-1])]
            out.register_hook(lambda g: seen[name].append(g.reshape(-1, g.shape[-1])))
        lin.register_forward_hook(hook)
    quantize = B.qlora_act_quantize
    B.qlora_act_quantize = lambda *a, **kw: made.append(1) or quantize(*a, **kw)
    try:
        res = []
        for model in (plain, block):
            x = case.X().to(DEV).requires_grad_(True)
            y = model(x)
            y.backward(case.grad().to(DEV))
            res.append((y, x.grad))
    finally:
        B.qlora_act_quantize = quantize
    assert len(made) == 3
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    for name in L.PROJECTIONS:
        lin = block.lin[name]
        assert torch.equal(plain.lin[name].B.grad, lin.B.grad)
        X, dY = seen[name]
        M.within(lin.A.grad, *_bound_dA(R.bf16_to_f64(dY), R.bf16_to_f64(lin.B), lin.scale,
                                             R.bf16_to_f64(X) if name == "o" else _restored(X)))

    seen.clear()
    for lin in block.lin.values():
        lin._forward_hooks.clear()
    held = []
    for model in (plain, block):
        x = case.X().to(DEV).requires_grad_(True)
        before = torch.cuda.memory_allocated()
        y = model(x)
        held.append(torch.cuda.memory_allocated() - before)
        del y
    # Two normed inputs and the MLP's: 1 + 2 / 64 bytes an element for 2.
    assert held[0] - held[1] >= 0.9 * 128 * (2 * 256 + 704) * (1 - 2 / 64), held


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
def test_decoder_block_of_many_adapters(keep8):
    """Every projection of the block with its own three adapters, one id a
    sequence: each adapter's gradients and the input's are those of the block
    with that adapter alone, run on that adapter's sequences."""
    case = WL.DecoderLayerCase(batch=3, seq=64, hidden=256, heads=4, mlp=704, r=16, alpha=32.0)
    base = L.build_decoder(case, torch.device(DEV))
    lins = {}
    for i, name in enumerate(L.PROJECTIONS):
        n, k = case.proj_shape(name)
        A = WL.bf16(WL.normal((3, 16, k), 0.02, 500 + i)).to(DEV)
        Bm = WL.bf16(WL.normal((3, n, 16), 0.02, 600 + i)).to(DEV)
        lins[name] = L.MultiQLoRALinear(base.lin[name].w, A, Bm, torch.full((3,), 2.0, device=DEV))
    block = L.DecoderLayer(case.heads, lins, act8=keep8)
    ids = torch.tensor([2, 0, 2], dtype=torch.int32, device=DEV)
    x = case.X().to(DEV).requires_grad_(True)
    y = block(x, ids)
    y.backward(case.grad().to(DEV))
    assert B.qlora_poll_device_error() == 0
    for a, rows in ((0, [1]), (2, [0, 2])):
        one = L.DecoderLayer(case.heads, {p: L.QLoRALinear(lins[p].w, lins[p].A[a].detach(), lins[p].B[a].detach(),
                                                           32.0) for p in L.PROJECTIONS}, act8=keep8)
        xa = case.X()[rows].to(DEV).requires_grad_(True)
        ya = one(xa)
        ya.backward(case.grad()[rows].to(DEV))
        # As test_layer: about a dozen bf16 roundings along the longest path on
        # each side, relative to the largest value.
        assert _rel(y[rows], ya) <= 2e-2 and _rel(x.grad[rows], xa.grad) <= 5e-2
        for p in L.PROJECTIONS:
            assert _rel(lins[p].A.grad[a], one.lin[p].A.grad) <= 5e-2
            assert _rel(lins[p].B.grad[a], one.lin[p].B.grad) <= 5e-2
    for p in L.PROJECTIONS:
        assert not lins[p].A.grad[1].any() and not lins[p].B.grad[1].any()


def _rel(got, ref):
    return float((got.detach().double() - ref.detach().double()).abs().max() / ref.detach().double().abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
def test_captured_training_step_follows_its_inputs(keep8):
    """Forward and backward of the module in one graph; new rows, ids and
    upstream gradients give what the uncaptured step gives on them."""
    c, d = (M.case(150, 264, 192, 16, 5, "mixed", seed) for seed in (390, 391))
    lin = _module(c, act8=keep8)
    X, ids, dY = c.X.to(DEV).requires_grad_(True), c.ids.to(DEV), c.dY.to(DEV)

    def step():
        Y = lin(X, ids)
        return (Y.detach(),) + torch.autograd.grad(Y, (X, lin.A, lin.B), dY)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for case in (d, c):
        with torch.no_grad():
            X.copy_(case.X), ids.copy_(case.ids), dY.copy_(case.dY)
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert B.qlora_poll_device_error() == 0
