"""Many adapters on one weight, on the CPU: pins of ``oracle/multi.py`` and the
entry points' argument checks (every call returns before the library's first
CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

from bit_nf4_quantized_qlora_b200 import binding as B
from oracle import linear, multi

P = 0x10000000
MIS = P + 8
MAX_SIZE = 2 ** 64 - 1


def _case(m=7, n=6, k=5, r=3, count=4, seed=0):
    g = np.random.default_rng(seed)
    f = g.standard_normal
    ids = np.array([2, -1, 0, 2, 9, 0, 3])[:m]
    return f((m, k)), f((n, k)), f((count, r, k)), f((count, n, r)), np.array([0.5, 1.0, 2.0, 0.25])[:count], ids, f((m, n))


def test_rows_equal_the_one_adapter_layer():
    X, W, A, Bm, s, ids, dY = _case()
    Y = multi.fwd(X, W, A, Bm, s, ids)
    for i, a in enumerate(ids):
        ok = 0 <= a < 4
        want = linear.fwd(X[i:i + 1], W, A[a], Bm[a], s[a]) if ok else linear.fwd(X[i:i + 1], W)
        assert np.allclose(Y[i], want[0], rtol=1e-13, atol=0)


def test_one_adapter_everywhere_is_the_layer():
    X, W, A, Bm, s, _, dY = _case()
    ids = np.full(7, 2)
    T = multi.lora_t(X, A, s, ids)
    dX, dA, dB = multi.bwd(dY, X, T, W, A, Bm, s, ids)
    rA, rB = linear.lora_grads(X, dY, A[2], Bm[2], s[2])
    assert np.allclose(dX, linear.bwd_dx(dY, W, A[2], Bm[2], s[2])) and np.allclose(dA[2], rA) and np.allclose(dB[2], rB)
    assert not dA[[0, 1, 3]].any() and not dB[[0, 1, 3]].any()


def test_gradients_by_finite_differences():
    X, W, A, Bm, s, ids, dY = _case(seed=3)
    T = multi.lora_t(X, A, s, ids)
    grads = multi.bwd(dY, X, T, W, A, Bm, s, ids)
    loss = lambda: float((multi.fwd(X, W, A, Bm, s, ids) * dY).sum())
    for v, g in zip((X, A, Bm), grads):
        num = np.zeros_like(v)
        for j in np.ndindex(v.shape):
            old = v[j]
            v[j] = old + 1e-5
            up = loss()
            v[j] = old - 1e-5
            num[j] = (up - loss()) / 2e-5
            v[j] = old
        assert np.max(np.abs(num - g)) <= 1e-7 * max(1.0, np.max(np.abs(g)))


# ---- argument checks --------------------------------------------------------


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def _w(n=1024, k=1024, codes=P):
    return B.NF4WeightC(codes, P, P, n, k, 64, 256)


def _set(A=P, Bm=P, scale=P, count=8, r=16):
    return B.AdapterSetC(A, Bm, scale, count, r)


def _fwd(lib, s=_set(), w=_w(), **a):
    return lib.qlora_linear_fwd_multi(a.get("X", P), a.get("m", 16), ctypes.byref(w), ctypes.byref(s) if s else None,
                                      a.get("ids", P), a.get("Y", P), a.get("ws", P), a.get("ws_bytes", 1 << 22), None)


def _bwd(lib, s=_set(), w=_w(), act=None, **a):
    return lib.qlora_linear_bwd_multi(a.get("dY", P), a.get("X", P), ctypes.byref(act) if act else None,
                                      a.get("T", P), a.get("m", 16), ctypes.byref(w), ctypes.byref(s) if s else None,
                                      a.get("ids", P), a.get("dX", P), a.get("dA", P), a.get("dB", P), a.get("ws", P),
                                      a.get("ws_bytes", 1 << 22), None)


@pytest.mark.parametrize("call", [_fwd, _bwd], ids=["fwd", "bwd"])
def test_bad_sets_and_ids_are_rejected(lib, call):
    assert call(lib, s=None) == call(lib, s=_set(A=0)) == call(lib, s=_set(Bm=0)) == B.QLORA_ERR_NULL
    assert call(lib, s=_set(scale=0)) == call(lib, ids=None) == call(lib, w=_w(codes=0)) == B.QLORA_ERR_NULL
    for bad in (_set(r=0), _set(r=24), _set(r=272), _set(r=-16), _set(count=0), _set(count=65536)):
        assert call(lib, s=bad) == B.QLORA_ERR_SHAPE
    assert call(lib, m=-1) == call(lib, m=(1 << 22) + 1) == B.QLORA_ERR_SHAPE
    assert call(lib, w=_w(k=1000)) == call(lib, w=_w(n=1020)) == B.QLORA_ERR_SHAPE
    assert call(lib, s=_set(A=MIS)) == call(lib, s=_set(scale=P + 2)) == call(lib, ids=P + 1) == B.QLORA_ERR_ALIGN
    assert call(lib, ws=None) == call(lib, ws_bytes=500) == B.QLORA_ERR_WORKSPACE
    assert call(lib, ws=MIS) == B.QLORA_ERR_ALIGN


def test_fwd_rejects_bad_tensors_and_takes_an_empty_batch(lib):
    assert _fwd(lib, X=None) == _fwd(lib, Y=None) == B.QLORA_ERR_NULL
    assert _fwd(lib, X=MIS) == _fwd(lib, Y=MIS) == B.QLORA_ERR_ALIGN
    assert _fwd(lib, m=0, X=None, Y=None, ids=None, ws=None) == B.QLORA_OK


def test_bwd_wants_one_input_and_T_with_a_checkpoint(lib):
    act = B.Act8C(P, P, 16, 1024)
    assert _bwd(lib, X=None) == _bwd(lib, act=act) == B.QLORA_ERR_NULL              # neither, both
    assert _bwd(lib, X=None, act=act, T=None) == B.QLORA_ERR_NULL
    assert _bwd(lib, X=None, act=B.Act8C(P, P, 17, 1024)) == B.QLORA_ERR_SHAPE
    assert _bwd(lib, X=None, act=B.Act8C(P, P, 16, 512)) == B.QLORA_ERR_SHAPE
    assert _bwd(lib, X=None, act=B.Act8C(MIS, P, 16, 1024)) == B.QLORA_ERR_ALIGN
    assert _bwd(lib, dY=None) == _bwd(lib, dA=None) == _bwd(lib, dB=None) == B.QLORA_ERR_NULL
    assert _bwd(lib, dY=MIS) == _bwd(lib, dX=MIS) == _bwd(lib, T=MIS) == B.QLORA_ERR_ALIGN


def test_workspace_sizes(lib):
    f = B.qlora_multi_workspace_bytes
    assert f(B.QLORA_OP_FWD, 16, 1024, 1024, 16, 8) == 512                          # T alone on the decode path
    assert f(B.QLORA_OP_FWD, 17, 1024, 1024, 16, 8) > f(B.QLORA_OP_FWD, 16, 1024, 1024, 16, 8)
    assert f(B.QLORA_OP_LORA_BWD, 0, 1024, 1024, 16, 8) == 0
    for bad in ((7, 16, 64, 64, 16, 1), (0, -1, 64, 64, 16, 1), (0, 16, 0, 64, 16, 1), (0, 16, 64, 64, 0, 1),
                (0, 16, 64, 64, 16, 0), (0, 16, 64, 64, 16, 65536), (0, (1 << 22) + 1, 64, 64, 16, 1)):
        assert f(*bad) == MAX_SIZE, bad


@pytest.mark.parametrize("m", [1, 63, 64, 65, 130, 1000])
@pytest.mark.parametrize("count", [1, 2, 9, 70])
def test_row_lists_fit_their_buffer(m, count):
    """The list layout: adapter a's list starts at 64 (floor(b / 64) + a), b
    the rows with a lower id, and is padded to whole 64s; lists never overlap
    and the last ends inside 64 (floor(m / 64) + count) entries."""
    g = np.random.default_rng(m * 100 + count)
    for _ in range(20):
        ids = g.integers(-1, count, size=m)
        end = 0
        for a in range(count):
            start = 64 * (int(((ids >= 0) & (ids < a)).sum()) // 64 + a)
            assert start >= end
            end = start + -(-int((ids == a).sum()) // 64) * 64
        assert end <= 64 * (m // 64 + count)


def test_binding_refuses_what_it_cannot_pass_on():
    bf = torch.bfloat16
    w = B.NF4Weight(torch.zeros(64 * 64 // 2, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8), torch.zeros(1), 64, 64)
    A, Bm = torch.zeros(2, 16, 64, dtype=bf), torch.zeros(2, 64, 16, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        B.qlora_linear_fwd_multi(torch.zeros(4, 64, dtype=bf), w, A, Bm, torch.ones(2), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="3-D"):
        B.qlora_linear_bwd_multi(torch.zeros(4, 64, dtype=bf), torch.zeros(4, 64, dtype=bf), w, A[0], Bm, torch.ones(2),
                                 torch.zeros(4, dtype=torch.int32))
