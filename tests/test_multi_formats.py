"""The many-adapter calls over every codebook and absmax format and at sizes of
real projections, against the defined weight W^ = bf16(level . constant).

For m <= 16 the kernels multiply bf16(g L + h), take h off and scale by c / g
(g >= 1, -1/8 < h <= 0) instead of rounding each product, so a weight differs
from W^ by at most

    H |W^| (1 + H)               W^'s own rounding, half a step
    H (|L| + |h| / g) |c|        the level's, with |h| / g < 1/8

The element-wise bound takes every rounding at its largest and the same sign.
The rms bound takes them as independent: a relative rounding of at most half a
step H is at most H / sqrt 3 in the mean square; Y's own, W^'s, the level's and
T's are four of them, each of no more than the value they round."""
import numpy as np
import pytest
import torch

import multi_refs as M
import oracle_refs as R
from bit_nf4_quantized_qlora_b200 import binding as B
from bit_nf4_quantized_qlora_b200 import workloads as WL
from oracle import nf4, quant

DEV = "cuda:0"
FORMATS = [(cb, dq) for cb in ("nf4", "fp4", "int4") for dq in ("linear8", "fp8_mean")]


def _bf16(x):
    return quant.bf16_bits_to_f32(quant.bf16_rne_bits(np.asarray(x, dtype=np.float32))).astype(np.float64)


def test_rounding_of_the_level_forms():
    """The constants are what their definition picks, and cost what is said of
    them: 0.06 % up to four rows and 0.08 % above, rms, where bf16(L) costs 0.14 %."""
    L = nf4.levels_f32().astype(np.float64)
    w = np.random.default_rng(0).standard_normal((4000, 64))
    c = np.abs(w).max(1, keepdims=True)
    code = np.abs((w / c)[..., None] - L).argmin(-1)
    often = np.bincount(code.ravel(), minlength=16) / code.size

    def rms(g, h):
        e = (_bf16(L * g + h) - h) / g - L
        return np.sqrt(((e[code] * c) ** 2).mean() / ((L[code] * c) ** 2).mean())

    def off(g, h):
        t = (L * g + h).astype(np.float32).astype(np.float64)
        return ((_bf16(t) - t) / g) ** 2

    h = -np.arange(256)[:, None] / 2048
    sums = np.stack([off(1 + i / 2048, h).sum(1) for i in range(2048)])
    assert np.unravel_index(sums.argmin(), sums.shape) == (1695, 97)
    assert (off(1 + np.arange(4096)[:, None] / 4096, 0.0) * often).sum(1).argmin() == 1789
    assert abs(rms(1.0, 0.0) - 1.4e-3) < 1e-4
    assert abs(rms(1 + 1695 / 2048, -97 / 2048) - 0.6e-3) < 0.5e-4
    assert abs(rms(1 + 1789 / 4096, 0.0) - 0.8e-3) < 0.5e-4


class Layer(M.Case):
    """A case whose W^ is the quantized weight's own, whatever its format."""

    def __post_init__(self):
        self.ids_np = self.ids.numpy()
        self.Xf, self.dYf, self.Af, self.Bf = (R.bf16_to_f64(t) for t in (self.X, self.dY, self.A, self.B))
        self.s = self.scale.double().numpy()

    def quantized(self, codebook="nf4", dq="linear8"):
        self.w = B.qlora_quantize_4bit_dq(self.W.to(DEV), B.CODEBOOKS[codebook], dq_format=B.DQ_FORMATS[dq])
        self.W_ = R.bf16_to_f64(B.qlora_dequant(self.w))
        return self

    def W_hat(self):
        return self.W_

    def check_small(self, Y):
        """m <= 16 against W^ (see the module's docstring)."""
        n, k = self.W_.shape
        r = self.A.shape[1]
        ref = M.multi.fwd(self.Xf, self.W_, self.Af, self.Bf, self.s, self.ids_np)
        # A block's constant is its largest magnitude up to 8 bits: |L| of the
        # largest element is 1 (FP4, INT4 and NF4 alike), so |c| <= max |W^| (1 + 2 H).
        c = np.repeat(np.abs(self.W_).reshape(n, k // 64, 64).max(2), 64, axis=1) * (1 + 2 * M.H)
        Xa, Aa, Ba = np.abs(self.Xf), np.abs(self.Af), np.abs(self.Bf)
        T = np.abs(M.multi.lora_t(self.Xf, self.Af, self.s, self.ids_np))
        Ta = M.multi.lora_t(Xa, Aa, self.s, self.ids_np)
        term, terma = M._through(T, Ba, self.ids_np), M._through(Ta, Ba, self.ids_np)
        Wa = np.abs(self.W_)
        tol = (M.H * np.abs(ref) + Xa @ (M.H * (1 + M.H) * (2 * Wa + c / 8)).T + M.H * (1 + M.H) * term
               + 2 * (k + r) * M.E * (Xa @ Wa.T + 2 * terma))
        M.within(Y, ref, tol * (1 + M.H))
        got = R.bf16_to_f64(Y)
        base = self.Xf @ self.W_.T
        parts = [np.mean(v ** 2) for v in (ref, base, base, ref - base)]
        assert np.mean((got - ref) ** 2) <= M.H ** 2 / 3 * sum(parts)


def layer(m, n, k, r, count, order, seed, codebook="nf4", dq="linear8"):
    g = np.random.default_rng(seed + 1)
    return Layer(WL.weight(n, k, 0.02, seed), WL.bf16(WL.normal((m, k), 1.0, seed + 2)),
                 WL.bf16(WL.normal((m, n), 1.0, seed + 3)), WL.bf16(WL.normal((count, r, k), 0.02, seed + 4)),
                 WL.bf16(WL.normal((count, n, r), 0.05, seed + 5)),
                 torch.from_numpy(g.choice([0.25, 0.5, 1.0, 2.0], size=count).astype(np.float32)),
                 torch.from_numpy(M.ids_for(m, count, order, seed + 6))).quantized(codebook, dq)


def _fwd(c):
    return B.qlora_linear_fwd_multi(c.X.to(DEV), c.w, *c.on(DEV))


def _check_bwd(c):
    T = WL.bf16(torch.from_numpy(M.multi.lora_t(c.Xf, c.Af, c.s, c.ids_np)).float())
    got = B.qlora_linear_bwd_multi(c.dY.to(DEV), c.X.to(DEV), c.w, *c.on(DEV), T=T.to(DEV))
    c.check_bwd(got, c.Xf, R.bf16_to_f64(T))


# The streaming kernel's three forms (k = 192, 1280, 1024 and 4096) up to four
# rows, the ring kernel above.
@pytest.mark.gpu
@pytest.mark.parametrize("codebook,dq", FORMATS)
@pytest.mark.parametrize("m,k", [(1, 192), (4, 1280), (1, 1024), (3, 4096), (4, 4096), (5, 192), (16, 1088), (12, 4096)])
def test_decode_forward_against_the_defined_weight(m, k, codebook, dq):
    c = layer(m, 264, k, 16, 3, "mixed", 16000 + m + k, codebook, dq)
    c.check_small(_fwd(c))
    assert B.qlora_poll_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("codebook,dq", FORMATS)
@pytest.mark.parametrize("m", [17, 130, 600])
def test_tiles_and_gradients_of_every_format(m, codebook, dq):
    c = layer(m, 264, 320, 32, 4, "mixed", 16100 + m, codebook, dq)
    c.check_fwd(_fwd(c))
    _check_bwd(c)
    assert B.qlora_poll_device_error() == 0


# A 7B model's attention projection and gate.
@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(4096, 4096), (11008, 4096)])
@pytest.mark.parametrize("m", [1, 4, 16])
def test_real_projections_decode(m, n, k):
    c = layer(m, n, k, 16, 8, "mixed", 16200 + m)
    c.check_small(_fwd(c))


@pytest.mark.gpu
@pytest.mark.parametrize("n,k,r,order", [(4096, 4096, 16, "mixed"), (4096, 11008, 64, "segments"), (11008, 4096, 64, "segments")])
def test_real_projections_prompts_and_gradients(n, k, r, order):
    c = layer(300, n, k, r, 8, order, 16300 + r)
    c.check_fwd(_fwd(c))
    _check_bwd(c)
    assert B.qlora_poll_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m,pad", [(1, 3), (3, 1), (2, 8), (9, 7), (12, 37)])
def test_padded_rows_of_nan_in_a_decode_batch(m, pad):
    """Rows without an adapter behind the live ones, NaN in X: the live rows are
    right and the padding's are NaN."""
    c = layer(m, 264, 1024, 16, 3, "segments", 16400 + m + pad)
    X = torch.cat([c.X, torch.full((pad, 1024), float("nan"), dtype=c.X.dtype)]).to(DEV)
    ids = torch.cat([c.ids, torch.full((pad,), -1, dtype=torch.int32)]).to(DEV)
    A, Bm, s, _ = c.on(DEV)
    Y = B.qlora_linear_fwd_multi(X, c.w, A, Bm, s, ids)
    c.check_small(Y[:m])
    assert bool(Y[m:].isnan().all())
