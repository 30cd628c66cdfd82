"""Inputs and element-wise bounds for the many-adapter and checkpoint tests.

The bounds are derived, per element: a bf16 rounding is off by at most
H = 2^-8 of the value; each of the terms of an fp32 sum adds at most 2^-24 of
the sum of magnitudes; rank-r intermediates (T, U) are rounded to bf16 once.
"""
from dataclasses import dataclass

import numpy as np
import torch

import oracle_refs as R
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import workloads as WL
from oracle import linear, multi, nf4, quant

H = 2.0 ** -8
E = 2.0 ** -24


def ids_for(m, count, order, seed):
    """int32 row ids: "one" (all adapter 0), "segments" (runs, shuffled, some
    empty), "mixed" (any order, some rows without an adapter, ids past both
    ends among them), "none" (no row has one), "last" (all the last adapter)."""
    g = np.random.default_rng(seed)
    if order == "one":
        return np.zeros(m, dtype=np.int32)
    if order == "last":
        return np.full(m, count - 1, dtype=np.int32)
    if order == "none":
        return np.full(m, -1, dtype=np.int32)
    if order == "segments":
        cuts = np.sort(g.integers(0, m + 1, size=count - 1))
        return g.permutation(count)[np.searchsorted(cuts, np.arange(m), side="right")].astype(np.int32)
    ids = g.integers(0, count, size=m)
    bad = np.array([-1, -7, count, count + 5, 2 ** 31 - 1, -2 ** 31])
    return np.where(g.random(m) < 0.15, g.choice(bad, size=m), ids).astype(np.int32)


@dataclass
class Case:
    W: torch.Tensor
    X: torch.Tensor
    dY: torch.Tensor
    A: torch.Tensor
    B: torch.Tensor
    scale: torch.Tensor
    ids: torch.Tensor

    def __post_init__(self):
        self.ids_np = self.ids.numpy()
        self.Xf, self.dYf, self.Af, self.Bf = (R.bf16_to_f64(t) for t in (self.X, self.dY, self.A, self.B))
        self.s = self.scale.double().numpy()
        self.packed, self.q, self.S = R.quantize(self.W)

    def weight(self, dev):
        return B.qlora_quantize_nf4_dq(self.W.to(dev))

    def W_hat(self):
        return quant.dequant_bf16_values(self.packed, self.q, self.S).reshape(self.W.shape)

    def W_stream(self):
        """The weight-streaming kernels' weight: bf16(g L + h) less h, scaled
        by c' / g after the product.  Up to four rows, the pair of g = 1 + i / 2048
        and h = -j / 2048, j < 256, that brings the levels closest to bf16 numbers;
        above, a factor g alone."""
        L = nf4.levels_f32()
        g, h = (1 + 1695 / 2048, -97 / 2048) if self.X.shape[0] <= 4 else (1 + 1789 / 4096, 0.0)
        scaled = (L.astype(np.float64) * g + h).astype(np.float32)
        lv = (quant.bf16_bits_to_f32(quant.bf16_rne_bits(scaled)).astype(np.float64) - h) / g
        c = np.repeat(quant.absmax_dequant(self.q, self.S).astype(np.float64), 64)
        return (lv[quant.unpack_codes(self.packed)] * c).reshape(self.W.shape)

    def on(self, dev):
        return tuple(t.to(dev) for t in (self.A, self.B, self.scale, self.ids))

    def check_fwd(self, Y):
        W = self.W_stream() if self.X.shape[0] <= 16 else self.W_hat()
        n, k = W.shape
        r = self.A.shape[1]
        ref = multi.fwd(self.Xf, W, self.Af, self.Bf, self.s, self.ids_np)
        Xa, Aa, Ba = np.abs(self.Xf), np.abs(self.Af), np.abs(self.Bf)
        T = np.abs(multi.lora_t(self.Xf, self.Af, self.s, self.ids_np))
        Ta = multi.lora_t(Xa, Aa, self.s, self.ids_np)
        # One rounding of T, its own accumulation, and the sum's.
        term, terma = _through(T, Ba, self.ids_np), _through(Ta, Ba, self.ids_np)
        tol = H * np.abs(ref) + H * (1 + H) * term + (k + r) * E * (Xa @ np.abs(W).T + 2 * terma)
        within(Y, ref, tol)

    def check_bwd(self, got, X, T):
        """got = (dX, dA, dB); X and T (fp64) as the call had them."""
        W = self.W_hat()
        n, k = W.shape
        m, r = self.X.shape[0], self.A.shape[1]
        rX, rA, rB = multi.bwd(self.dYf, X, T, W, self.Af, self.Bf, self.s, self.ids_np)
        Ya, Aa, Ba, Xa = np.abs(self.dYf), np.abs(self.Af), np.abs(self.Bf), np.abs(X)
        dX, dA, dB = got
        if dX is not None:
            tol = H * np.abs(rX) + (n + r) * E * (Ya @ np.abs(W))
            for a in range(self.A.shape[0]):
                i = multi.rows_of(self.ids_np, a)
                U, Ua = np.abs(linear.lora_u(self.dYf[i], self.Bf[a], self.s[a])), linear.lora_u(Ya[i], Ba[a], self.s[a])
                tol[i] += H * (1 + H) * (U @ Aa[a]) + 2 * (n + r) * E * (Ua @ Aa[a])
            within(dX, rX, tol)
        tA, tB = H * np.abs(rA), H * np.abs(rB)
        for a in range(self.A.shape[0]):
            i = multi.rows_of(self.ids_np, a)
            U, Ua = np.abs(linear.lora_u(self.dYf[i], self.Bf[a], self.s[a])), linear.lora_u(Ya[i], Ba[a], self.s[a])
            tA[a] += H * (1 + H) * (U.T @ Xa[i]) + 2 * (n + m) * E * (Ua.T @ Xa[i])
            tB[a] += m * E * (Ya[i].T @ np.abs(T[i]))
        within(dA, rA, tA)
        within(dB, rB, tB)


def _through(T, Ba, ids):
    out = np.zeros((T.shape[0], Ba.shape[1]))
    for a in range(Ba.shape[0]):
        i = multi.rows_of(ids, a)
        out[i] = T[i] @ Ba[a].T
    return out


def within(got, ref, tol):
    g = R.bf16_to_f64(got)
    assert g.shape == ref.shape
    assert np.all(np.isfinite(g))
    over = np.abs(g - ref) - tol
    assert over.size == 0 or over.max() <= 0, f"{(over > 0).mean():.2%} of the elements off, worst by {over.max():.3e}"


def case(m, n, k, r, count, order, seed, zero_weight=False):
    """Adapters whose term is of the frozen product's size; scales of both signs'
    magnitudes 1/4 .. 2."""
    W = torch.zeros(n, k) if zero_weight else WL.weight(n, k, 0.02, seed)
    g = np.random.default_rng(seed + 1)
    return Case(W, WL.bf16(WL.normal((m, k), 1.0, seed + 2)), WL.bf16(WL.normal((m, n), 1.0, seed + 3)),
                WL.bf16(WL.normal((count, r, k), 0.02, seed + 4)), WL.bf16(WL.normal((count, n, r), 0.05, seed + 5)),
                torch.from_numpy(g.choice([0.25, 0.5, 1.0, 2.0], size=count).astype(np.float32)),
                torch.from_numpy(ids_for(m, count, order, seed + 6)))
