"""Sizes that no call takes: the workspace query and the modules name them."""
import pytest
import torch

from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import layer as L

MAX_SIZE = 2 ** 64 - 1


@pytest.mark.parametrize("op", [B.QLORA_OP_FWD, B.QLORA_OP_LORA_BWD])
def test_workspace_bytes_of_sizes_no_call_takes(op):
    f = B.qlora_multi_workspace_bytes
    assert 0 < f(op, 40, 72, 128, 16, 3) < MAX_SIZE
    for m, n, k, r, count in ((40, 72, 128, 17, 3), (40, 72, 128, 272, 3), (40, 72, 128, 999, 3), (40, 72, 60, 16, 3),
                              (40, 72, 100, 16, 3), (40, 70, 128, 16, 3), (40, 72, 128, -16, 3),
                              (40, 1 << 32, 128, 16, 3), (40, 72, 1 << 32, 16, 3)):
        assert f(op, m, n, k, r, count) == MAX_SIZE, (m, n, k, r, count)


def test_the_binding_lets_the_call_name_such_sizes():
    """Without a workspace the binding asks for one; a rank no call takes must
    not become an allocation."""
    ws, size = B._multi_workspace(B.QLORA_OP_FWD, 40, 72, 128, 272, 3, None, torch.device("cpu"), None)
    assert size == 0


def test_modules_refuse_ranks_no_call_takes():
    w = B.NF4Weight(None, None, None, 24, 64)
    for r in (0, 8, 24, 272):
        with pytest.raises(ValueError, match="rank"):
            L.MultiQLoRALinear(w, torch.zeros(2, r, 64), torch.zeros(2, 24, r), torch.ones(2))
    with pytest.raises(ValueError, match="rank"):
        L.MultiQLoRALinear.from_adapters(w, [(torch.zeros(260, 64), torch.zeros(24, 260), 1.0)])
    with pytest.raises(ValueError, match="rank"):
        L.MultiQLoRALinear.from_adapters(w, [(torch.zeros(0, 64), torch.zeros(24, 0), 1.0)])
    with pytest.raises(ValueError, match="adapter"):
        L.MultiQLoRALinear.from_adapters(w, [])
    for A, Bm, s in ((torch.zeros(2, 16, 128), torch.zeros(2, 24, 16), torch.ones(2)),
                     (torch.zeros(2, 16, 64), torch.zeros(3, 24, 16), torch.ones(2)),
                     (torch.zeros(2, 16, 64), torch.zeros(2, 24, 16), torch.ones(3)),
                     (torch.zeros(16, 64), torch.zeros(24, 16), torch.ones(1))):
        with pytest.raises(ValueError, match="shape"):
            L.MultiQLoRALinear(w, A, Bm, s)


def test_an_adapter_whose_halves_do_not_fit_is_refused():
    """Padding would hide columns of B that no row of A feeds."""
    w = B.NF4Weight(None, None, None, 24, 64)
    ok = (torch.ones(8, 64), torch.ones(24, 8), 16.0)
    for bad in ((torch.ones(8, 64), torch.ones(24, 16), 16.0), (torch.ones(16, 64), torch.ones(24, 8), 16.0),
                (torch.ones(8, 128), torch.ones(24, 8), 16.0), (torch.ones(8, 64), torch.ones(32, 8), 16.0)):
        with pytest.raises(ValueError, match="adapter 1"):
            L.MultiQLoRALinear.from_adapters(w, [ok, bad])
