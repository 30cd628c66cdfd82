"""Cases, plain forms and exact values of the layer's operators for many
adapters on one frozen 4-bit weight and for 8-bit activation checkpoints.

    fwd_multi   Y[i] = X[i] W^T + s_a (X[i] A_a^T) B_a^T,  a = ids[i]
    bwd_multi   dX[i] = dY[i] W + s_a (dY[i] B_a) A_a,
                dA_a = s_a sum_i (dY[i] B_a)^T X[i],  dB_a = sum_i dY[i]^T T[i]
                over the rows i of adapter a; T is kept from the forward
    act8        X -> 8-bit codes and one bf16 scale per 64 values -> X again
    bwd_act8    the one-adapter backward with X read from its 8-bit codes
    train       fwd_multi, the 8-bit checkpoint of X, then bwd_multi from it

A row whose id lies outside [0, na) has no adapter.  The frozen weight is NF4
with double-quantized block constants.
"""
import math
from statistics import NormalDist

import torch

own = False

BLOCK, GROUP = 64, 256
DEV = "cuda"

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def _case(name, op, m, n, k, r=16, na=1, order="mixed", act=False):
    c = {"op": op, "m": m, "n": n, "k": k, "r": r, "na": na, "order": order, "act": act}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One request decoding through a 7B attention projection; eight adapters are loaded.
        _case("decode_m1_7b_attn", "fwd_multi", 1, 4096, 4096, 16, 8),
        # Sixteen requests decoding through the 7B gate, (nearly) every one with its own adapter.
        _case("decode_m16_7b_gate", "fwd_multi", 16, 11008, 4096, 16, 16),
        # A full decode batch on the 70B up-projection, 64 adapters and a few rows without one.
        _case("decode_m128_70b_up", "fwd_multi", 128, 28672, 8192, 16, 64),
        # Six prompts of odd lengths through the 7B down projection.
        _case("prefill_m1111_7b_down", "fwd_multi", 1111, 4096, 11008, 64, 6, "segments"),
        # Training eight tenants on the 7B gate, batch 4 x 1024 tokens packed tenant by tenant.
        _case("bwd_m4096_7b_gate", "bwd_multi", 4096, 11008, 4096, 64, 8, "segments"),
        # Tenants interleaved token by token: the order that packs worst.
        _case("bwd_m2000_mixed", "bwd_multi", 2000, 4096, 4096, 16, 32),
        # A ragged little batch: sizes inside one tile, a rank that is no power of two.
        _case("bwd_m130_ragged", "bwd_multi", 130, 520, 1088, 48, 5),
        # A micro-batch's activation checkpoint, and the training batch's.
        _case("act8_m17_4096", "act8", 17, 0, 4096),
        _case("act8_m8192_11008", "act8", 8192, 0, 11008),
        # The 7B down projection, whose input is the widest checkpoint of the block; a short odd batch.
        _case("bwd_act8_m4096_7b_down", "bwd_act8", 4096, 4096, 11008, 64),
        _case("bwd_act8_m300_7b_attn", "bwd_act8", 300, 4096, 4096, 16),
        # A whole step of four tenants on the 70B up-projection with the checkpoint in 8 bits.
        _case("train_m2048_70b_up", "train", 2048, 28672, 8192, 16, 4, "segments", True),
    ]


_TOP = 2048 * 28672 * 8192


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd_multi", "fwd_multi", "bwd_multi", "bwd_multi", "act8", "bwd_act8", "train"])
    while True:
        m = _log(rng, 1, 8192)
        n = 8 * max(1, _log(rng, 64, 28672) // 8)
        k = 64 * max(1, _log(rng, 64, 11008) // 64)
        if m * n * k <= _TOP:
            break
    r = rng.choice([16, 16, 32, 48, 64, 64, 128, 256])
    na = _log(rng, 1, 64)
    order = rng.choice(["segments", "mixed"])
    if op == "act8":
        return _case(None, op, m, 0, k)
    if op == "bwd_act8":
        return _case(None, op, m, n, k, r)
    act = op == "train" or (op == "bwd_multi" and rng.random() < 0.3)
    return _case(None, op, m, n, k, r, na, order, act)


def work(case):
    m, n, k, r, na = (case[x] for x in ("m", "n", "k", "r", "na"))
    if case["op"] == "act8":
        # X in; codes, scales and the restored X out.
        return {"bytes": 2 * m * k + (m * k + m * k // 32) + 2 * m * k, "flops": 0}
    w = n * k // 2 + n * k // BLOCK + 4 * ((n * k + BLOCK * GROUP - 1) // (BLOCK * GROUP))
    ids = 4 * m if case["op"] != "bwd_act8" else 0
    ad = 2 * r * (n + k) * min(na, m)
    fwd = {"bytes": w + 2 * m * (n + k) + ad + ids, "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    x = (m * k + m * k // 32) if case["act"] or case["op"] == "bwd_act8" else 2 * m * k
    bwd = {"bytes": w + 2 * m * (n + k) + x + 2 * m * r + ad + 2 * r * (n + k) * na + ids,
           "flops": 2 * m * n * k + 4 * m * r * (n + k)}
    if case["op"] == "fwd_multi":
        return fwd
    if case["op"] == "train":
        # Both passes, plus the checkpoint; the weight, adapters and ids are read again by the second pass.
        return {"bytes": fwd["bytes"] + bwd["bytes"] + m * k + m * k // 32, "flops": fwd["flops"] + bwd["flops"]}
    return bwd


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------


def _nf4_levels():
    """The sixteen NF4 levels: normal quantiles, 8 above zero, 7 below, zero."""
    nd = NormalDist()
    o = 1.0 - 0.5 * (1.0 / 32 + 1.0 / 30)
    pos = [nd.inv_cdf(o + (0.5 - o) * i / 8) for i in range(8)]
    neg = [-nd.inv_cdf(o + (0.5 - o) * i / 7) for i in range(7)]
    top = nd.inv_cdf(o)
    return sorted([v / top for v in pos + neg] + [0.0])


def _quantize_nf4(W, level):
    """Block codes (two per byte), 8-bit block constants and their group maxima."""
    n, k = W.shape
    c = W.view(-1, BLOCK).abs().amax(1)
    mid = (level[1:] + level[:-1]) * 0.5
    codes = torch.empty(n * k // 2, dtype=torch.uint8, device=W.device)
    step = 1 << 20
    for b in range(0, c.numel(), step):
        x = W.view(-1, BLOCK)[b:b + step] / c[b:b + step, None]
        q = torch.bucketize(x, mid, out_int32=True).view(-1, 2)
        codes[b * 32:b * 32 + q.shape[0]] = (q[:, 0] * 16 + q[:, 1]).to(torch.uint8)
    ng = (c.numel() + GROUP - 1) // GROUP
    pad = torch.zeros(ng * GROUP, device=W.device)
    pad[:c.numel()] = c
    S = pad.view(ng, GROUP).amax(1)
    q = torch.round(pad.view(ng, GROUP) / S[:, None] * 255.0).view(-1)[:c.numel()].to(torch.uint8)
    return codes, q.contiguous(), S.contiguous()


def _ids(case, g):
    m, na = case["m"], case["na"]
    if case["order"] == "segments":
        # One run of rows per adapter, in a shuffled order, of random lengths.
        cuts = torch.sort(torch.randint(0, m + 1, (na - 1,), device=DEV, generator=g)).values
        which = torch.bucketize(torch.arange(m, device=DEV), cuts, right=True)
        ids = torch.randperm(na, device=DEV, generator=g)[which]
    else:
        # Any adapter on any row; one row in sixteen has none.
        ids = torch.randint(0, na, (m,), device=DEV, generator=g)
        ids = torch.where(torch.rand(m, device=DEV, generator=g) < 1.0 / 16, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32)


def _act_quantize(X):
    """Codes int8 [m, k] and bf16 scales [m, k/64] of a bf16 X."""
    m, k = X.shape
    x = X.float().view(m, k // BLOCK, BLOCK)
    sc = (x.abs().amax(2) / 127.0).to(torch.bfloat16)
    s = sc.float()[:, :, None]
    q = torch.where(s > 0, torch.round(x / s), torch.zeros_like(x)).clamp(-127, 127)
    return q.view(m, k).to(torch.int8), sc


def _act_values(q, sc):
    m, k = q.shape
    return (q.float().view(m, k // BLOCK, BLOCK) * sc.float()[:, :, None]).view(m, k).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    m, n, k, r, na, op = (case[x] for x in ("m", "n", "k", "r", "na", "op"))

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device=DEV, generator=g) * std).to(torch.bfloat16)

    st = {"case": case, "X": normal(m, k)}
    # A few channels carry most of the magnitude, as a block's activations do.
    hot = torch.randint(0, k, (max(1, k // 256),), device=DEV, generator=g)
    st["X"][:, hot] *= 8.0
    if op == "act8":
        return _with_buffers(st)
    level = torch.tensor(_nf4_levels(), dtype=torch.float32, device=DEV)
    W = torch.randn(n, k, device=DEV, generator=g) * 0.02
    st["codes"], st["absmax_q"], st["group_scale"] = _quantize_nf4(W, level)
    del W
    st["level"] = level
    # Trained adapters: the low-rank term is of the base product's size.
    st["A"] = normal(na, r, k, std=0.02)
    st["B"] = normal(na, n, r, std=0.05)
    st["scale"] = torch.tensor([0.25, 0.5, 1.0, 2.0], device=DEV)[
        torch.randint(0, 4, (na,), device=DEV, generator=g)].contiguous()
    st["ids"] = _ids(case, g) if op != "bwd_act8" else torch.zeros(m, dtype=torch.int32, device=DEV)
    st["dY"] = normal(m, n, std=0.01)
    if op in ("bwd_multi", "bwd_act8"):
        # What a training step keeps from its forward.
        st["T"] = _adapter_in(st, st["X"].float()).to(torch.bfloat16)
        if case["act"] or op == "bwd_act8":
            st["q"], st["sc"] = _act_quantize(st["X"])
            del st["X"]
    st["s0"] = float(st["scale"][0])
    return _with_buffers(st)


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------


def _weight(st):
    """The frozen weight's values, bf16(level x constant), in 32 bits."""
    n, k = st["case"]["n"], st["case"]["k"]
    q = st["absmax_q"].float()
    t = (st["group_scale"] / 255.0).repeat_interleave(GROUP)[:q.numel()]
    c = q * t
    W = torch.empty(n * k, device=DEV)
    step = 1 << 20
    for b in range(0, c.numel(), step):
        byte = st["codes"][b * 32:(b + step) * 32]
        idx = torch.stack([byte >> 4, byte & 15], 1).view(-1, BLOCK).int()
        v = st["level"][idx] * c[b:b + step, None]
        W[b * BLOCK:(b + step) * BLOCK] = v.to(torch.bfloat16).float().view(-1)
    return W.view(n, k)


def _rows_of(st):
    """Per adapter: the rows that use it, as a column of ones and zeros."""
    for a in range(st["case"]["na"]):
        yield a, (st["ids"] == a).float()[:, None]


def _adapter_in(st, Xf):
    """s_a X A_a^T of every row's own adapter."""
    T = torch.zeros(Xf.shape[0], st["case"]["r"], device=DEV)
    for a, on in _rows_of(st):
        T += (Xf @ st["A"][a].float().t()) * (st["scale"][a] * on)
    return T


def _plain_fwd(st, W):
    Xf = st["X"].float()
    Y = Xf @ W.t()
    T = _adapter_in(st, Xf)
    for a, on in _rows_of(st):
        Y += (T * on) @ st["B"][a].float().t()
    return Y.to(torch.bfloat16), T


def _plain_bwd(st, W, Xf, T):
    dYf = st["dY"].float()
    dX = dYf @ W
    dA = torch.empty(st["A"].shape, dtype=torch.bfloat16, device=DEV)
    dB = torch.empty(st["B"].shape, dtype=torch.bfloat16, device=DEV)
    for a, on in _rows_of(st):
        U = (dYf @ st["B"][a].float()) * (st["scale"][a] * on)
        dX += U @ st["A"][a].float()
        dA[a] = (U.t() @ Xf).to(torch.bfloat16)
        dB[a] = (dYf.t() @ (T * on)).to(torch.bfloat16)
    return dX.to(torch.bfloat16), dA, dB


def _run_plain(st):
    op = st["case"]["op"]
    if op == "act8":
        return {"X": _act_values(*_act_quantize(st["X"]))}
    W = _weight(st)
    if op == "fwd_multi":
        return {"Y": _plain_fwd(st, W)[0]}
    if op == "train":
        Y, T = _plain_fwd(st, W)
        dX, dA, dB = _plain_bwd(st, W, _act_values(*_act_quantize(st["X"])).float(), T)
        return {"Y": Y, "dX": dX, "dA": dA, "dB": dB}
    Xf = _act_values(st["q"], st["sc"]).float() if "q" in st else st["X"].float()
    dX, dA, dB = _plain_bwd(st, W, Xf, st["T"].float())
    return {"dX": dX, "dA": dA, "dB": dB}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------


def _with_buffers(st):
    if own:
        from bit_nf4_quantized_qlora_b200 import binding as Q
        st["own"] = _buffers(st, Q)
    return st


def _buffers(st, Q):
    """What a program keeps between calls: the weight's handle, outputs and a workspace."""
    c = st["case"]
    m, n, k, r, na, op = (c[x] for x in ("m", "n", "k", "r", "na", "op"))

    def bf16(*shape):
        return torch.empty(*shape, dtype=torch.bfloat16, device=DEV)

    b = {}
    if op in ("act8", "train"):
        b["act"] = Q.Act8.empty(m, k, DEV)
    if op == "act8":
        b["X"] = bf16(m, k)
        return b
    b["w"] = Q.NF4Weight(st["codes"], st["absmax_q"], st["group_scale"], n, k)
    if op in ("fwd_multi", "train"):
        b["Y"] = bf16(m, n)
        b["wsf"] = torch.empty(max(16, Q.qlora_multi_workspace_bytes(Q.QLORA_OP_FWD, m, n, k, r, na)),
                               dtype=torch.uint8, device=DEV)
    if op != "fwd_multi":
        b["dX"] = bf16(m, k)
        b["dA"], b["dB"] = (bf16(r, k), bf16(n, r)) if op == "bwd_act8" else (bf16(na, r, k), bf16(na, n, r))
        need = (Q.qlora_workspace_bytes(Q.QLORA_OP_LORA_BWD, m, n, k, r) if op == "bwd_act8"
                else Q.qlora_multi_workspace_bytes(Q.QLORA_OP_LORA_BWD, m, n, k, r, na))
        b["ws"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    if op in ("bwd_multi", "bwd_act8") and "q" in st:
        b["act"] = Q.Act8(st["q"], st["sc"], m, k)
    return b


def _run_own(st):
    from bit_nf4_quantized_qlora_b200 import binding as Q
    b, op = st["own"], st["case"]["op"]
    if op == "act8":
        Q.qlora_act_quantize(st["X"], out=b["act"])
        return {"X": Q.qlora_act_dequant(b["act"], out=b["X"])}
    m, r = st["case"]["m"], st["case"]["r"]
    if op == "bwd_act8":
        dX, dA, dB = Q.qlora_linear_bwd_act8(st["dY"], b["act"], b["w"], st["A"][0], st["B"][0], r, st["s0"], st["T"],
                                             dX=b["dX"], dA=b["dA"], dB=b["dB"], ws=b["ws"])
        return {"dX": dX, "dA": dA[None], "dB": dB[None]}
    out = {}
    T, X = st.get("T"), b.get("act", st.get("X"))
    if op in ("fwd_multi", "train"):
        out["Y"] = Q.qlora_linear_fwd_multi(st["X"], b["w"], st["A"], st["B"], st["scale"], st["ids"], out=b["Y"],
                                            ws=b["wsf"])
        if op == "fwd_multi":
            return out
        Q.qlora_act_quantize(st["X"], out=b["act"])
        T = b["wsf"][:2 * m * r].view(torch.bfloat16).view(m, r)
    out["dX"], out["dA"], out["dB"] = Q.qlora_linear_bwd_multi(st["dY"], X, b["w"], st["A"], st["B"], st["scale"],
                                                               st["ids"], T=T, dX=b["dX"], dA=b["dA"], dB=b["dB"],
                                                               ws=b["ws"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# Exact values
# ---------------------------------------------------------------------------


def exact(case, seed):
    """The operators' definitions in 64 bits, row groups taken by index."""
    st = prepare(case, seed)
    m, n, k, r, na, op = (case[x] for x in ("m", "n", "k", "r", "na", "op"))

    def restored(q, sc):
        # The value an 8-bit code stands for is a bf16 number.
        v = q.double() * sc.double().repeat_interleave(BLOCK, 1)
        return v.to(torch.bfloat16).double()

    def codes_of(X):
        x = X.double()
        sc = torch.stack([x[:, b:b + BLOCK].abs().max(1).values / 127 for b in range(0, k, BLOCK)], 1).to(torch.bfloat16)
        wide = sc.double().repeat_interleave(BLOCK, 1)
        q = torch.zeros_like(x)
        live = wide > 0
        q[live] = torch.round(x[live] / wide[live]).clamp(-127, 127)
        return q, sc

    if op == "act8":
        return {"X": restored(*codes_of(st["X"]))}

    # The weight's values are bf16 numbers: the level times the 32-bit block constant, rounded.
    c = (st["absmax_q"].float() * (st["group_scale"] / torch.tensor(255.0, device=DEV))
         [torch.arange(n * k // BLOCK, device=DEV) // GROUP]).view(n, k // BLOCK)
    nib = torch.empty(n, k, dtype=torch.uint8, device=DEV)
    nib[:, 0::2] = (st["codes"] >> 4).view(n, k // 2)
    nib[:, 1::2] = (st["codes"] & 15).view(n, k // 2)
    W = torch.empty(n, k, dtype=torch.float64, device=DEV)
    for i in range(0, n, 1024):
        lv = st["level"].double()[nib[i:i + 1024].long()]
        W[i:i + 1024] = (lv * c[i:i + 1024].double().repeat_interleave(BLOCK, 1)).float().to(torch.bfloat16).double()
    rows = [torch.nonzero(st["ids"] == a)[:, 0] for a in range(na)]
    A, B, s = st["A"].double(), st["B"].double(), st["scale"].double()
    out = {}
    X = restored(st["q"], st["sc"]) if "q" in st else st["X"].double()
    if op in ("fwd_multi", "train"):
        T = torch.zeros(m, r, dtype=torch.float64, device=DEV)
        Y = torch.matmul(X, W.t())
        for a in range(na):
            T[rows[a]] = s[a] * torch.matmul(X[rows[a]], A[a].t())
            Y[rows[a]] = Y[rows[a]] + torch.matmul(T[rows[a]], B[a].t())
        out["Y"] = Y
        if op == "fwd_multi":
            return out
        X = restored(*codes_of(st["X"]))
    else:
        T = st["T"].double()
    dY = st["dY"].double()
    dX = torch.matmul(dY, W)
    dA = torch.zeros(na, r, k, dtype=torch.float64, device=DEV)
    dB = torch.zeros(na, n, r, dtype=torch.float64, device=DEV)
    for a in range(na):
        i = rows[a]
        U = s[a] * torch.matmul(dY[i], B[a])
        dX[i] = dX[i] + torch.matmul(U, A[a])
        dA[a] = torch.matmul(U.t(), X[i])
        dB[a] = torch.matmul(dY[i].t(), T[i])
    out["dX"], out["dA"], out["dB"] = dX, dA, dB
    return out
