"""Calls on another stream than the current one: what a call allocates (its
workspace, its outputs) comes from the pool of the stream it launches on.
Memory of the current stream's pool would go back to it when the call returns,
while the call's kernels still run, and could still be in use there when they
start.  The CPU tests watch the allocations through fakes; nothing is launched."""
import contextlib
import types

import pytest
import torch

import multi_refs as M
from bit_nf4_quantized_qlora_b200 import binding as B

DEV = "cuda:0"
M_, N_, K_, R_, COUNT = 24, 72, 128, 16, 3
HANDLE = 0x7F00


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _calls():
    """name -> call(stream) of every entry point that can allocate, on CPU tensors."""
    w = B.NF4Weight(torch.zeros(N_ * K_ // 2, dtype=torch.uint8), torch.zeros(N_ * K_ // 64, dtype=torch.uint8),
                    torch.zeros(2), N_, K_)
    X, dY, A, Bm, T = _bf(M_, K_), _bf(M_, N_), _bf(R_, K_), _bf(N_, R_), _bf(M_, R_)
    As, Bs, s, ids = _bf(COUNT, R_, K_), _bf(COUNT, N_, R_), torch.ones(COUNT), torch.zeros(M_, dtype=torch.int32)
    act = B.Act8(torch.zeros(M_, K_, dtype=torch.int8), _bf(M_, K_ // 64), M_, K_)
    return {
        "quantize": lambda st: B.qlora_quantize_nf4_dq(torch.zeros(N_, K_), stream=st),
        "dequant": lambda st: B.qlora_dequant(w, stream=st),
        "merge": lambda st: B.qlora_merge_adapter(w, A, Bm, R_, 1.0, want_f32=True, stream=st),
        "fwd": lambda st: B.qlora_linear_fwd(X, w, A, Bm, R_, 1.0, stream=st),
        "bwd_dx": lambda st: B.qlora_linear_bwd_dx(dY, w, A, Bm, R_, 1.0, stream=st),
        "lora_bwd": lambda st: B.qlora_lora_bwd(X, dY, A, Bm, R_, 1.0, stream=st),
        "bwd": lambda st: B.qlora_linear_bwd(dY, X, w, A, Bm, R_, 1.0, stream=st),
        "dropout": lambda st: B.qlora_lora_dropout(X, 0.5, 1, 2, stream=st),
        "fwd_dropout": lambda st: B.qlora_linear_fwd_dropout(X, w, A, Bm, R_, 1.0, 0.5, 1, 2, stream=st),
        "bwd_dx_dropout": lambda st: B.qlora_linear_bwd_dx_dropout(dY, w, A, Bm, R_, 1.0, 0.5, 1, 2, stream=st),
        "fwd_noalloc": lambda st: B.qlora_linear_fwd_noalloc(X, w, A, Bm, R_, 1.0, stream=st),
        "act_quantize": lambda st: B.qlora_act_quantize(X, stream=st),
        "act_dequant": lambda st: B.qlora_act_dequant(act, stream=st),
        "bwd_act8": lambda st: B.qlora_linear_bwd_act8(dY, act, w, A, Bm, R_, 1.0, T, stream=st),
        "fwd_multi": lambda st: B.qlora_linear_fwd_multi(X, w, As, Bs, s, ids, stream=st),
        "bwd_multi": lambda st: B.qlora_linear_bwd_multi(dY, X, w, As, Bs, s, ids, stream=st),
    }


@pytest.fixture
def watched(monkeypatch):
    """Fakes in place of CUDA: `seen` holds, for every allocation, the stream
    that was current."""
    seen, current = [], [None]

    @contextlib.contextmanager
    def stream(s):
        old, current[0] = current[0], s
        yield
        current[0] = old

    def noting(make):
        def f(*a, **kw):
            seen.append(current[0])
            return make(*a, **kw)
        return f

    real = B.lib()

    class Fake:
        def __getattr__(self, name):
            if name.endswith("workspace_bytes"):
                return getattr(real, name)
            return lambda *a: B.QLORA_OK

    monkeypatch.setattr(B, "lib", lambda: Fake())
    monkeypatch.setattr(B, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(B, "_stream_on", lambda device, stream: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noting(torch.empty_like))
    return seen


@pytest.mark.parametrize("name", sorted(_calls()))
def test_allocations_belong_to_the_calls_stream(watched, name):
    _calls()[name](HANDLE)
    assert watched and all(s == ("external", HANDLE) for s in watched)


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handles(watched, handle):
    """0 and 1 are the default stream's handles, not an external stream's."""
    _calls()["fwd_multi"](handle)
    assert watched and all(s == "default" for s in watched)


def test_without_a_stream_allocations_stay_on_the_current_one(watched):
    for call in _calls().values():
        call(None)
    assert watched and all(s is None for s in watched)


@pytest.mark.gpu
@pytest.mark.parametrize("as_handle", [False, True])
def test_results_while_the_current_stream_allocates(as_handle):
    """Every call on a side stream without buffers, the current stream filling
    blocks of the same sizes in between, gives what it gives with buffers kept."""
    c = M.case(700, 264, 1088, 32, 6, "mixed", 12000)
    A, Bm, s, ids = c.on(DEV)
    w, X, dY = c.weight(DEV), c.X.to(DEV), c.dY.to(DEV)
    size = (700, 264, 1088, 32, 6)
    ws = torch.empty(max(B.qlora_multi_workspace_bytes(op, *size) for op in (B.QLORA_OP_FWD, B.QLORA_OP_LORA_BWD)),
                     dtype=torch.uint8, device=DEV)
    want = [t.clone() for t in (B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, ws=ws),
                                *B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids, ws=ws))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    st = side.cuda_stream if as_handle else side
    for _ in range(10):
        got = [B.qlora_linear_fwd_multi(X, w, A, Bm, s, ids, stream=st)]
        junk = [torch.full((ws.numel(),), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
        got += B.qlora_linear_bwd_multi(dY, X, w, A, Bm, s, ids, stream=st)
        junk += [torch.full_like(g, float("nan")) for g in got]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk, got
    assert B.qlora_poll_device_error() == 0
