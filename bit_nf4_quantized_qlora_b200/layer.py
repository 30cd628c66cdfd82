"""The QLoRA linear layer as a torch autograd function, and the 7B-shaped
decoder block used to measure it inside a transformer layer.

The frozen base weight is held only in its NF4 + double-quant form and the
adapters A [r x k], B [n x r] are bf16 parameters ("QLoRA and Quantized
Training", The idea; "QLoRA", Follow one QLoRA training step): the forward is
one ``qlora_linear_fwd`` and the backward one ``qlora_linear_bwd`` (input
gradient and adapter gradients, reusing the forward's rank-r intermediate),
all in libqlora's kernels.  Two variations of it: the input kept for the
backward as an 8-bit checkpoint (``act8``), and one frozen weight under the
adapters of many tenants, one named per row (``MultiQLoRALinear``; "QLoRA",
Training setup versus deployment setup).  The rest of the decoder block (RMSNorm, causal
attention, SiLU gating, residual adds) is plain PyTorch: it is not part of
the quantized layer, and the pages leave it to the host framework.
"""
from typing import Dict, Optional, Sequence, Tuple, Union

import torch
import torch.nn.functional as F

from . import binding as B


def _kept_T(ws: torch.Tensor, m: int, r: int) -> Optional[torch.Tensor]:
    # The forward leaves T = bf16(s X A^T) at the start of its workspace;
    # the backward takes it instead of recomputing it.
    return ws[:m * r * 2].view(torch.bfloat16).view(m, r) if r > 0 and m > 0 else None


def _checkpoint_of(act: B.Act8, X: torch.Tensor) -> B.Act8:
    if (act.m, act.k) != tuple(X.shape):
        raise ValueError(f"the checkpoint holds [{act.m} x {act.k}], the input is {list(X.shape)}")
    return act


class QLoRALinearFunction(torch.autograd.Function):
    """Y = X . dequant(W)^T + s (X A^T) B^T for X [m x k] (bf16, contiguous)."""

    @staticmethod
    def forward(ctx, X: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, w: B.NF4Weight, r: int, scale: float):
        m = X.shape[0]
        ws = torch.empty(max(1, B.qlora_workspace_bytes(B.QLORA_OP_FWD, m, w.n, w.k, r)), dtype=torch.uint8,
                         device=X.device)
        Y = B.qlora_linear_fwd(X, w, A, Bm, r, scale, ws=ws)
        ctx.save_for_backward(X, A, Bm, _kept_T(ws, m, r))
        ctx.w, ctx.r, ctx.scale = w, r, scale
        return Y

    @staticmethod
    def backward(ctx, dY: torch.Tensor):
        X, A, Bm, T = ctx.saved_tensors
        dY = dY.contiguous()
        dX, dA, dB = B.qlora_linear_bwd(dY, X, ctx.w, A, Bm, ctx.r, ctx.scale, T=T,
                                        want_dx=ctx.needs_input_grad[0])
        return dX, dA, dB, None, None, None


class QLoRALinearAct8Function(torch.autograd.Function):
    """The same Y; X is not kept, its 8-bit checkpoint `act` is (1.03 bytes an
    element for 2).  dX and dB are as with X, dA = s (dY B)^T X^."""

    @staticmethod
    def forward(ctx, X: torch.Tensor, act: B.Act8, A: torch.Tensor, Bm: torch.Tensor, w: B.NF4Weight, r: int,
                scale: float):
        m = X.shape[0]
        ws = torch.empty(max(1, B.qlora_workspace_bytes(B.QLORA_OP_FWD, m, w.n, w.k, r)), dtype=torch.uint8,
                         device=X.device)
        Y = B.qlora_linear_fwd(X, w, A, Bm, r, scale, ws=ws)
        ctx.save_for_backward(act.codes, act.scale, A, Bm, _kept_T(ws, m, r))
        ctx.w, ctx.r, ctx.scale, ctx.shape = w, r, scale, (act.m, act.k)
        return Y

    @staticmethod
    def backward(ctx, dY: torch.Tensor):
        codes, scale, A, Bm, T = ctx.saved_tensors
        dX, dA, dB = B.qlora_linear_bwd_act8(dY.contiguous(), B.Act8(codes, scale, *ctx.shape), ctx.w, A, Bm, ctx.r,
                                             ctx.scale, T, want_dx=ctx.needs_input_grad[0])
        return dX, None, dA, dB, None, None, None


class MultiQLoRALinearFunction(torch.autograd.Function):
    """Y[i] = X[i] . dequant(W)^T + s_a (X[i] A_a^T) B_a^T, a = ids[i]; an id
    outside [0, count) takes no adapter.  With a checkpoint `act` of X, that is
    kept in X's place."""

    @staticmethod
    def forward(ctx, X: torch.Tensor, act: Optional[B.Act8], A: torch.Tensor, Bm: torch.Tensor, scale: torch.Tensor,
                ids: torch.Tensor, w: B.NF4Weight):
        m, count, r = X.shape[0], A.shape[0], A.shape[1]
        ws = torch.empty(B.qlora_multi_workspace_bytes(B.QLORA_OP_FWD, m, w.n, w.k, r, count), dtype=torch.uint8,
                         device=X.device)
        Y = B.qlora_linear_fwd_multi(X, w, A, Bm, scale, ids, ws=ws)
        kept = (X,) if act is None else (act.codes, act.scale)
        ctx.save_for_backward(A, Bm, scale, ids, _kept_T(ws, m, r), *kept)
        ctx.w, ctx.shape = w, tuple(X.shape)
        return Y

    @staticmethod
    def backward(ctx, dY: torch.Tensor):
        A, Bm, scale, ids, T, *kept = ctx.saved_tensors
        X = kept[0] if len(kept) == 1 else B.Act8(*kept, *ctx.shape)
        dX, dA, dB = B.qlora_linear_bwd_multi(dY.contiguous(), X, ctx.w, A, Bm, scale, ids, T=T,
                                              want_dx=ctx.needs_input_grad[0])
        return dX, None, dA, dB, None, None, None


class QLoRALinear(torch.nn.Module):
    """A frozen NF4 weight [n x k] with trainable bf16 adapters (rank r, s = alpha / r).

    With `act8` the input is kept for the backward in 8 bits; layers that share
    an input share one checkpoint through `act` (``qlora_act_quantize`` of the
    input as [rows x k])."""

    def __init__(self, w: B.NF4Weight, A: torch.Tensor, Bm: torch.Tensor, alpha: float, act8: bool = False):
        super().__init__()
        self.w = w
        self.act8 = act8
        self.r = A.shape[0]
        self.scale = alpha / self.r
        self.A = torch.nn.Parameter(A.to(torch.bfloat16).contiguous())
        self.B = torch.nn.Parameter(Bm.to(torch.bfloat16).contiguous())

    @classmethod
    def from_float(cls, W: torch.Tensor, A: torch.Tensor, Bm: torch.Tensor, alpha: float,
                   codebook: int = B.QLORA_CODEBOOK_NF4, act8: bool = False) -> "QLoRALinear":
        """Quantize an fp32 weight [n x k] on its device (libqlora's quantize
        kernel), NF4 unless another codebook (B.QLORA_CODEBOOK_*) is named."""
        return cls(B.qlora_quantize_4bit_dq(W.float().contiguous(), codebook), A, Bm, alpha, act8)

    @torch.no_grad()
    def merged_weight(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """W' = W^ + s . B . A [n x k] (bf16 or fp32) for export or serving
        without the adapter (libqlora's merge kernel)."""
        want_f32 = dtype == torch.float32
        h, f = B.qlora_merge_adapter(self.w, self.A.detach(), self.B.detach(), self.r, self.scale,
                                     want_bf16=not want_f32, want_f32=want_f32)
        return f if want_f32 else h

    def forward(self, x: torch.Tensor, act: Optional[B.Act8] = None) -> torch.Tensor:
        lead = x.shape[:-1]
        X = x.reshape(-1, x.shape[-1]).contiguous()
        if (self.act8 or act is not None) and torch.is_grad_enabled():
            act = B.qlora_act_quantize(X.detach()) if act is None else _checkpoint_of(act, X)
            y = QLoRALinearAct8Function.apply(X, act, self.A, self.B, self.w, self.r, self.scale)
        else:
            y = QLoRALinearFunction.apply(X, self.A, self.B, self.w, self.r, self.scale)
        return y.reshape(*lead, self.w.n)


class MultiQLoRALinear(torch.nn.Module):
    """One frozen NF4 weight [n x k] under the trainable bf16 adapters of many
    tenants: A [count x r x k], B [count x n x r], s = alpha / rank of each.

    ``forward(x, ids)`` takes int32 ids on x's device, one per row of x
    (x.shape[:-1]) or one per leading index (one per sequence of a [batch x
    tokens x k] input); an id outside [0, count) means the frozen weight alone.
    `act8` and `act` as in ``QLoRALinear``.  In a captured step the ids may
    change between replays; graphs that autograd built outside the capture from
    the same parameters must be gone before it starts."""

    def __init__(self, w: B.NF4Weight, A: torch.Tensor, Bm: torch.Tensor, scale: torch.Tensor, act8: bool = False):
        super().__init__()
        if A.dim() != 3 or A.shape[2] != w.k or Bm.shape != (A.shape[0], w.n, A.shape[1]) or scale.shape != A.shape[:1]:
            raise ValueError(f"A, B and scale of shape {list(A.shape)}, {list(Bm.shape)} and {list(scale.shape)} are no "
                             f"adapters of a [{w.n} x {w.k}] weight")
        if not 0 < A.shape[1] <= 256 or A.shape[1] % 16:
            raise ValueError(f"the adapters' rank must be a multiple of 16 up to 256, not {A.shape[1]}")
        self.w = w
        self.act8 = act8
        self.A = torch.nn.Parameter(A.to(torch.bfloat16).contiguous())
        self.B = torch.nn.Parameter(Bm.to(torch.bfloat16).contiguous())
        self.register_buffer("scale", scale.to(torch.float32).contiguous())

    def _apply(self, fn, recurse=True):
        # The scales are fp32 in a model of any type; they only change device.
        scale = self.scale
        super()._apply(fn, recurse)
        if self.scale.dtype != torch.float32:
            self.scale = scale.to(self.scale.device)
        return self

    @classmethod
    def from_adapters(cls, w: B.NF4Weight, adapters: Sequence[Tuple[torch.Tensor, torch.Tensor, float]],
                      act8: bool = False) -> "MultiQLoRALinear":
        """Adapters (A [r_a x k], B [n x r_a], alpha_a) of any ranks up to 256,
        padded with zeros to the largest (a multiple of 16)."""
        ranks = [A.shape[0] for A, _, _ in adapters]
        if not ranks or not 0 < min(ranks) <= max(ranks) <= 256:
            raise ValueError(f"one or more adapters of ranks 1 to 256 are needed, not {ranks}")
        for i, (A, Bm, _) in enumerate(adapters):
            if A.shape[1:] != (w.k,) or Bm.shape != (w.n, A.shape[0]):
                raise ValueError(f"adapter {i} of shapes {list(A.shape)} and {list(Bm.shape)} does not fit a "
                                 f"[{w.n} x {w.k}] weight")
        r = -(-max(ranks) // 16) * 16
        As = torch.stack([F.pad(A.to(torch.bfloat16), (0, 0, 0, r - A.shape[0])) for A, _, _ in adapters])
        Bs = torch.stack([F.pad(Bm.to(torch.bfloat16), (0, r - Bm.shape[1])) for _, Bm, _ in adapters])
        scale = torch.tensor([alpha / A.shape[0] for A, _, alpha in adapters], dtype=torch.float32, device=As.device)
        return cls(w, As, Bs, scale, act8)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, act: Optional[B.Act8] = None) -> torch.Tensor:
        lead = x.shape[:-1]
        X = x.reshape(-1, x.shape[-1]).contiguous()
        if ids is None:
            raise ValueError("a layer of many adapters needs the rows' ids")
        if ids.shape != lead[:ids.dim()]:
            raise ValueError(f"ids of shape {list(ids.shape)} do not lead rows of shape {list(lead)}")
        rows = ids.reshape(ids.shape + (1,) * (len(lead) - ids.dim())).expand(lead).reshape(-1).contiguous()
        if not torch.is_grad_enabled():
            act = None
        elif act is not None:
            _checkpoint_of(act, X)
        elif self.act8:
            act = B.qlora_act_quantize(X.detach())
        y = MultiQLoRALinearFunction.apply(X, act, self.A, self.B, self.scale, rows, self.w)
        return y.reshape(*lead, self.w.n)


RMS_EPS = 1e-5
PROJECTIONS = ("q", "k", "v", "o", "gate", "up", "down")


def rms_norm(x: torch.Tensor, eps: float = RMS_EPS) -> torch.Tensor:
    xf = x.float()
    return (xf * torch.rsqrt(xf.pow(2).mean(-1, keepdim=True) + eps)).to(x.dtype)


class DecoderLayer(torch.nn.Module):
    """Pre-norm decoder block with seven QLoRA projections: attention
    (q, k, v, o; causal, no positional rotation) and a SwiGLU MLP
    (gate, up, down).  The RMSNorm gains are 1 (frozen).

    With projections of many adapters, all or some of the seven,
    ``forward(x, ids)`` passes those the ids.
    With `act8` the projections keep their inputs in 8 bits, one checkpoint for
    q, k and v and one for gate and up.  o keeps its bf16 input, which
    attention's own backward holds in any case."""

    def __init__(self, heads: int, linears: Dict[str, Union[QLoRALinear, MultiQLoRALinear]], act8: bool = False):
        super().__init__()
        self.heads = heads
        self.act8 = act8
        self.lin = torch.nn.ModuleDict(linears)

    def _project(self, names: Sequence[str], x: torch.Tensor, ids: Optional[torch.Tensor], act8: bool):
        kw = {}
        if act8 and torch.is_grad_enabled():
            kw["act"] = B.qlora_act_quantize(x.detach().reshape(-1, x.shape[-1]).contiguous())
        lins = [self.lin[name] for name in names]
        return [lin(x, ids, **kw) if isinstance(lin, MultiQLoRALinear) else lin(x, **kw) for lin in lins]

    def forward(self, x: torch.Tensor, ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        b, t, h = x.shape
        d = h // self.heads
        q, k, v = (y.view(b, t, self.heads, d).transpose(1, 2)
                   for y in self._project(("q", "k", "v"), rms_norm(x), ids, self.act8))
        att = F.scaled_dot_product_attention(q, k, v, is_causal=True)
        x = x + self._project(("o",), att.transpose(1, 2).reshape(b, t, h), ids, False)[0]
        g, u = self._project(("gate", "up"), rms_norm(x), ids, self.act8)
        return x + self._project(("down",), F.silu(g) * u, ids, self.act8)[0]


def build_decoder(case, device: torch.device, act8: bool = False) -> DecoderLayer:
    """Quantize the seven fp32 weights of a decoder workload (see
    ``workloads.DecoderLayerCase``) on `device` and attach its adapters."""
    lins = {}
    for name in PROJECTIONS:
        lins[name] = QLoRALinear.from_float(case.W(name).to(device), case.A(name).to(device),
                                            case.B(name).to(device), case.alpha)
    return DecoderLayer(case.heads, lins, act8)


def linear_flops(case, tokens: int) -> Dict[str, float]:
    """Algorithmic FLOPs of the seven quantized projections for `tokens` rows:
    forward 2mnk + 2mr(n+k), input gradient the same, adapter gradients
    2mr(n+2k) + 2mnr."""
    fwd = bwd = grads = 0.0
    for name in PROJECTIONS:
        n, k = case.proj_shape(name)
        m, r = tokens, case.r
        fwd += 2 * m * n * k + 2 * m * r * (n + k)
        bwd += 2 * m * n * k + 2 * m * r * (n + k)
        grads += 2 * m * r * (n + 2 * k) + 2 * m * n * r
    return {"fwd": fwd, "bwd_dx": bwd, "lora_grads": grads, "total": fwd + bwd + grads}
