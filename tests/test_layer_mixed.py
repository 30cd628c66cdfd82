"""A decoder block whose projections are partly of many adapters and partly of
one: the row ids go to those that take them."""
import pytest
import torch

from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import layer as L
from bit_nf4_quantized_qlora_b200 import workloads as WL

DEV = "cuda:0"
MANY = ("q", "v")


def _stub_block(monkeypatch, act8, grads):
    """A block on the CPU whose layer calls note what they get: X . 0 plus the ids' presence."""
    hidden, mlp, heads = 64, 128, 2
    seen = {}

    def one(X, A, Bm, w, r, scale):
        seen.setdefault(w, []).append(("one", None, None))
        return X.new_zeros(X.shape[0], w.n)

    def one8(X, act, A, Bm, w, r, scale):
        seen.setdefault(w, []).append(("one", None, act))
        return X.new_zeros(X.shape[0], w.n)

    def many(X, act, A, Bm, scale, ids, w):
        seen.setdefault(w, []).append(("many", ids, act))
        return X.new_zeros(X.shape[0], w.n)

    class W(B.NF4Weight):
        __hash__ = object.__hash__

    monkeypatch.setattr(L.QLoRALinearFunction, "apply", one)
    monkeypatch.setattr(L.QLoRALinearAct8Function, "apply", one8)
    monkeypatch.setattr(L.MultiQLoRALinearFunction, "apply", many)
    monkeypatch.setattr(B, "qlora_act_quantize", lambda X: B.Act8(None, None, *X.shape))
    lins, weights = {}, {}
    for name in L.PROJECTIONS:
        n, k = (mlp, hidden) if name in ("gate", "up") else (hidden, mlp) if name == "down" else (hidden, hidden)
        weights[name] = W(None, None, None, n, k)
        if name in MANY:
            lins[name] = L.MultiQLoRALinear(weights[name], torch.zeros(3, 16, k), torch.zeros(3, n, 16), torch.ones(3))
        else:
            lins[name] = L.QLoRALinear(weights[name], torch.zeros(16, k), torch.zeros(n, 16), 32.0)
    block = L.DecoderLayer(heads, lins, act8=act8)
    with torch.set_grad_enabled(grads):
        y = block(torch.ones(2, 5, hidden, dtype=torch.bfloat16), torch.tensor([2, 0], dtype=torch.int32))
    assert y.shape == (2, 5, hidden)
    return {name: seen[weights[name]] for name in L.PROJECTIONS}


@pytest.mark.parametrize("grads", [True, False])
@pytest.mark.parametrize("act8", [False, True])
def test_ids_go_to_the_projections_that_take_them(monkeypatch, act8, grads):
    seen = _stub_block(monkeypatch, act8, grads)
    for name, calls in seen.items():
        (kind, ids, act), = calls
        assert kind == ("many" if name in MANY else "one")
        if kind == "many":
            assert ids.tolist() == [2] * 5 + [0] * 5
        assert (act is not None) == (act8 and grads and name != "o")


@pytest.mark.gpu
@pytest.mark.parametrize("keep8", [False, True])
def test_mixed_block_against_blocks_of_one_adapter(keep8):
    """Each sequence's outputs and gradients are those of a block with its
    tenant's adapters on q and v; the shared adapters' gradients are the sum."""
    case = WL.DecoderLayerCase(batch=3, seq=64, hidden=256, heads=4, mlp=704, r=16, alpha=32.0)
    base = L.build_decoder(case, torch.device(DEV))
    lins = {}
    for i, name in enumerate(L.PROJECTIONS):
        if name in MANY:
            n, k = case.proj_shape(name)
            A = WL.bf16(WL.normal((2, 16, k), 0.02, 700 + i)).to(DEV)
            Bm = WL.bf16(WL.normal((2, n, 16), 0.02, 800 + i)).to(DEV)
            lins[name] = L.MultiQLoRALinear(base.lin[name].w, A, Bm, torch.full((2,), 2.0, device=DEV))
        else:
            lins[name] = base.lin[name]
    block = L.DecoderLayer(case.heads, lins, act8=keep8)
    x = case.X().to(DEV).requires_grad_(True)
    y = block(x, torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV))
    y.backward(case.grad().to(DEV))
    with torch.no_grad():
        assert torch.equal(block(x, torch.tensor([1, 0, 1], dtype=torch.int32, device=DEV)), y)
    shared = {p: [lins[p].A.grad.double(), lins[p].B.grad.double()] for p in L.PROJECTIONS if p not in MANY}
    total = {p: [torch.zeros_like(t) for t in ts] for p, ts in shared.items()}
    for a, rows in ((0, [1]), (1, [0, 2])):
        one = L.DecoderLayer(case.heads, {p: L.QLoRALinear(lins[p].w, lins[p].A[a].detach() if p in MANY else lins[p].A.detach(),
                                                           lins[p].B[a].detach() if p in MANY else lins[p].B.detach(), 32.0)
                                          for p in L.PROJECTIONS}, act8=keep8)
        xa = case.X()[rows].to(DEV).requires_grad_(True)
        ya = one(xa)
        ya.backward(case.grad()[rows].to(DEV))
        # As test_layer: about a dozen bf16 roundings along the longest path on
        # each side, relative to the largest value.
        assert _rel(y[rows], ya) <= 2e-2 and _rel(x.grad[rows], xa.grad) <= 5e-2
        for p in L.PROJECTIONS:
            if p in MANY:
                assert _rel(lins[p].A.grad[a], one.lin[p].A.grad) <= 5e-2
                assert _rel(lins[p].B.grad[a], one.lin[p].B.grad) <= 5e-2
            else:
                total[p][0] += one.lin[p].A.grad.double()
                total[p][1] += one.lin[p].B.grad.double()
    for p, (gA, gB) in shared.items():
        assert _rel(gA, total[p][0]) <= 5e-2 and _rel(gB, total[p][1]) <= 5e-2


def _rel(got, ref):
    return float((got.detach().double() - ref.detach().double()).abs().max() / ref.detach().double().abs().max())


def test_a_layer_of_many_adapters_names_missing_ids():
    lin = L.MultiQLoRALinear(B.NF4Weight(None, None, None, 24, 64), torch.zeros(2, 16, 64), torch.zeros(2, 24, 16),
                             torch.ones(2))
    with pytest.raises(ValueError, match="ids"):
        lin(torch.zeros(2, 64, dtype=torch.bfloat16), None)
