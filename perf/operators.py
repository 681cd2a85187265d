"""Operators of the weight-only 4-bit layer, for measurement: plain forms and the library's calls.

Three operators, told apart by ``case["op"]``:

``quant``  the offline quantiser (smoothing folded in, group scales) and the values its codes stand for;
``gemm``   x [M, K] times 4-bit weights [N, K] with group scales, for a few tokens;
``moe``    a whole mixture-of-experts layer for a few tokens (router, top-k, gated experts, weighted sum).

The packed format: K is cut into blocks of 128 (the last one padded), 64 bytes each; the code of
k = 128 b + 32 w + 8 t + i (w, t < 4, i < 8) is nibble i // 2 + 4 (i % 2) of the little-endian 32-bit word at
byte 64 b + 16 t + 4 w of its row.  Scales are bf16 [ceil(K / G), N], zero points uint8 of the same shape (absent: 8),
and a code stands for (code - zero) * scale.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SHIFTS = [4 * (i // 2) + 16 * (i % 2) for i in range(8)]


# ------------------------------------------------------------------------------------------------ cases
def listed():
    q = dict(op="quant")
    g = dict(op="gemm")
    m = dict(op="moe")
    return [
        # offline: a small ragged fp32 layer (short last group, short last block)
        dict(q, name="quant_1040x1000_f32_g32", K=1040, N=1000, dt="f32", group=32, asym=False),
        # offline: the fused gate and up projection of an 8B-class layer, zero points, group 64
        dict(q, name="quant_4096x28672_bf16_g64z", K=4096, N=28672, dt="bf16", group=64, asym=True),
        # one user's decode step, 8B-class: fused QKV (latency counts)
        dict(g, name="gemm_m1_6144x4096", M=1, N=6144, K=4096, dt="bf16", group=128, asym=False),
        # one user's decode step, 8B-class: the down projection (long K)
        dict(g, name="gemm_m1_4096x14336", M=1, N=4096, K=14336, dt="bf16", group=128, asym=False),
        # a ragged fp32 layer: a few tokens, short last group and block, odd N
        dict(g, name="gemm_m3_1001x1040_f32_g32z", M=3, N=1001, K=1040, dt="f32", group=32, asym=True),
        # a small decode batch on a 175B-class output projection, zero points, group 64
        dict(g, name="gemm_m7_12288x12288_g64z", M=7, N=12288, K=12288, dt="bf16", group=64, asym=True),
        # decode batches of an 8B-class model: fused gate and up at 16 tokens, output projection at 64
        dict(g, name="gemm_m16_28672x4096", M=16, N=28672, K=4096, dt="bf16", group=128, asym=False),
        dict(g, name="gemm_m64_4096x4096", M=64, N=4096, K=4096, dt="bf16", group=128, asym=False),
        # one user's decode step: many small experts (latency counts), and few large ones (bandwidth)
        dict(m, name="moe_t1_e128k8_2048x768", T=1, E=128, top_k=8, D=2048, F=768, dt="bf16", group=128, asym=False,
             renorm=True),
        dict(m, name="moe_t1_e8k2_4096x14336", T=1, E=8, top_k=2, D=4096, F=14336, dt="bf16", group=128, asym=False,
             renorm=True),
        # a ragged fp32 layer with an odd number of experts, weights not renormalised
        dict(m, name="moe_t5_e9k3_1040x720_f32_g32z", T=5, E=9, top_k=3, D=1040, F=720, dt="f32", group=32, asym=True,
             renorm=False),
        # a decode batch over many small experts: nearly every expert has a few tokens
        dict(m, name="moe_t32_e128k8_2048x768_g64", T=32, E=128, top_k=8, D=2048, F=768, dt="bf16", group=64,
             asym=False, renorm=True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "moe", "moe"])
    c = dict(op=op, dt=rng.choice(["bf16", "bf16", "f32"]), group=rng.choice([32, 64, 128]),
             asym=rng.choice([False, True]))
    if op == "quant":
        c["K"] = _log(rng, 256, 14336, 16)
        c["N"] = _log(rng, 64, min(28672, 4096 * 28672 // c["K"]), 8)
    elif op == "gemm":
        c["M"] = _log(rng, 1, 64)
        c["K"] = _log(rng, 256, 14336, 16)
        c["N"] = _log(rng, 64, min(28672, 12288 * 12288 // c["K"]))
    else:
        c["T"] = _log(rng, 1, 32)
        c["E"] = _log(rng, 4, 128)
        c["top_k"] = rng.randint(1, min(8, c["E"]))
        c["D"] = _log(rng, 256, 4096, 16)
        c["F"] = _log(rng, 128, min(14336, max(128, 128 * 2048 * 768 // (c["E"] * c["D"]))), 16)
        c["renorm"] = rng.choice([False, True])
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _pack(codes):
    """Codes [..., K] (integers 0 .. 15) -> packed rows [..., 64 ceil(K / 128)] uint8."""
    K = codes.shape[-1]
    codes = torch.nn.functional.pad(codes, (0, -K % 128)).to(torch.int64)
    v = codes.unflatten(-1, (-1, 4, 4, 8))  # block, w, t, i
    word = (v << torch.tensor(_SHIFTS, device=codes.device)).sum(-1)  # block, w, t
    return word.transpose(-1, -2).to(torch.int32).flatten(-3).contiguous().view(torch.uint8)


def _weights(gen, K, N, group, asym):
    """A packed weight [N, K] as a quantiser leaves one of normally distributed values: codes, scales, zero points."""
    G = -(-K // group)
    v = torch.randn(N, K, generator=gen, device=DEV) * 2.6
    sg = (0.02 / 2.6 * (0.8 + 0.4 * torch.rand(G, N, generator=gen, device=DEV))).to(torch.bfloat16)
    if not asym:
        return _pack((v.round().clamp(-7, 7) + 8).to(torch.uint8)), sg, None
    zp = torch.randint(6, 10, (G, N), generator=gen, device=DEV, dtype=torch.uint8)
    v = v.round() + zp.repeat_interleave(group, 0)[:K].T
    return _pack(v.clamp(0, 15).to(torch.uint8)), sg, zp


def _activations(gen, M, K, dt):
    """Smoothed activations: normal, with about 1% of the channels some times larger, the same for every token."""
    x = torch.randn(M, K, generator=gen, device=DEV)
    big = torch.rand(K, generator=gen, device=DEV) < 0.01
    return (x * torch.where(big, 10.0, 1.0)).to(_DT[dt])


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    op, group, asym = case["op"], case["group"], case["asym"]
    st = dict(case)
    if op == "quant":
        K, N = case["K"], case["N"]
        st["W"] = (torch.randn(K, N, generator=gen, device=DEV) * 0.02).to(_DT[case["dt"]])
        st["s"] = 0.5 + 2.0 * torch.rand(K, generator=gen, device=DEV)
    elif op == "gemm":
        st["wq"], st["sg"], st["zp"] = _weights(gen, case["K"], case["N"], group, asym)
        st["x"] = _activations(gen, case["M"], case["K"], case["dt"])
    else:
        D, F, E = case["D"], case["F"], case["E"]
        up = [_weights(gen, D, 2 * F, group, asym) for _ in range(E)]
        down = [_weights(gen, F, D, group, asym) for _ in range(E)]
        for k, parts in (("13", up), ("2", down)):
            st["w" + k] = torch.stack([p[0] for p in parts])
            st["s" + k] = torch.stack([p[1] for p in parts])
            st["z" + k] = torch.stack([p[2] for p in parts]) if asym else None
        st["x"] = _activations(gen, case["T"], D, case["dt"])
        st["wr"] = (torch.randn(E, D, generator=gen, device=DEV) * (1.5 / math.sqrt(D))).to(_DT[case["dt"]])
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _values(wq, sg, zp, K, group):
    """Packed weights [..., N, row bytes] -> the values they stand for, [..., N, K] in binary32."""
    shifts = torch.tensor(_SHIFTS, device=wq.device, dtype=torch.int32)
    q = (wq.view(torch.int32).unflatten(-1, (-1, 4, 4)).unsqueeze(-1) >> shifts) & 15  # block, t, w, i
    q = q.transpose(-2, -3).flatten(-4)[..., :K]
    at = torch.arange(K, device=wq.device) // group
    zero = 8.0 if zp is None else zp.transpose(-1, -2)[..., at].float()
    return (q.float() - zero) * sg.transpose(-1, -2)[..., at].float()


def _plain_quant(st):
    K, N, group = st["K"], st["N"], st["group"]
    w = st["W"].float() * st["s"][:, None]
    w = torch.nn.functional.pad(w, (0, 0, 0, -K % group)).view(-1, group, N)  # padding is 0: no max, no min changes
    if st["asym"]:
        lo, hi = w.amin(1).clamp(max=0.0), w.amax(1).clamp(min=0.0)
        sg = ((hi - lo) / 15.0).to(torch.bfloat16)
        d = torch.where(sg == 0, 1.0, sg.float())
        zp = torch.where(sg == 0, 0.0, (-lo / d).round().clamp(0, 15))
        q = ((w / d[:, None]).round() + zp[:, None]).clamp(0, 15) - zp[:, None]
    else:
        sg = (w.abs().amax(1) / 7.0).to(torch.bfloat16)
        d = torch.where(sg == 0, 1.0, sg.float())
        zp = None
        q = (w / d[:, None]).round().clamp(-7, 7)
    v = (q * sg.float()[:, None]).flatten(0, 1)[:K].T.contiguous().to(_DT[st["dt"]])
    return {"values": v, "scales": sg} | ({} if zp is None else {"zeros": zp.to(torch.uint8)})


def _plain_gemm(st):
    w = _values(st["wq"], st["sg"], st["zp"], st["K"], st["group"])
    return (st["x"].float() @ w.T).to(_DT[st["dt"]])


def _plain_moe(st):
    T, E, k, F = st["T"], st["E"], st["top_k"], st["F"]
    x = st["x"].float()
    logits = st["x"].double() @ st["wr"].double().T  # values next to a border decide who is chosen
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    p = torch.softmax(logits, -1).gather(1, order)
    if st["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    used, at = torch.unique(order, return_inverse=True)
    pick = lambda a: None if a is None else a[used]  # noqa: E731
    w13 = _values(pick(st["w13"]), pick(st["s13"]), pick(st["z13"]), st["D"], st["group"])
    gu = torch.einsum("td,end->ten", x, w13)
    del w13
    h = gu[..., :F] * torch.sigmoid(gu[..., :F]) * gu[..., F:]
    share = torch.zeros(T, len(used), device=x.device).scatter_(1, at, p.float())
    w2 = _values(pick(st["w2"]), pick(st["s2"]), pick(st["z2"]), F, st["group"])
    y = torch.einsum("tef,edf->td", h * share[..., None], w2)
    return {"y": y.to(_DT[st["dt"]]), "ids": order.int(), "weights": p.float()}


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        import w8a8_smoothquant_gemm_b200 as sq
        group, dt = state["group"], _DT[state["dt"]]
        if state["op"] == "quant":
            wq, sg, zp, _, _ = sq.sq_fold_quant_weights_w4(state["W"], state["s"], group=group, asym=state["asym"])
            v = sq.sq_w4_dequant(wq, sg, zp, K=state["K"], group=group, out_dtype=dt)
            return {"values": v, "scales": sg} | ({} if zp is None else {"zeros": zp})
        if state["op"] == "gemm":
            return sq.sq_w4_gemm(state["x"], state["wq"], state["sg"], state["zp"], group=group, out_dtype=dt)
        if "workspace" not in state:  # a user's program keeps one for all its calls
            state["workspace"] = sq.sq_moe_w4_workspace(state["T"], state["D"], state["F"], state["E"], state["top_k"])
        y, ids, wts = sq.sq_moe_w4(state["x"], state["wr"], state["top_k"], state["w13"], state["s13"], state["w2"],
                                   state["s2"], z13=state["z13"], z2=state["z2"], group=group, renorm=state["renorm"],
                                   out_dtype=dt, workspace=state["workspace"])
        return {"y": y, "ids": ids, "weights": wts}
    return {"quant": _plain_quant, "gemm": _plain_gemm, "moe": _plain_moe}[state["op"]](state)


def work(case):
    op, group, e = case["op"], case["group"], 2 if case["dt"] == "bf16" else 4
    side = 3 if case["asym"] else 2  # bytes beside each group's codes

    def packed(K, N):
        return N * K // 2 + -(-K // group) * N * side

    if op == "quant":  # the weights and factors in; the codes out and in again; the values they stand for out
        K, N = case["K"], case["N"]
        return {"bytes": 2 * K * N * e + 4 * K + 2 * packed(K, N), "flops": 4 * K * N}
    if op == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": packed(K, N) + (M * K + M * N) * e, "flops": 2 * M * N * K}
    T, E, k, D, F = case["T"], case["E"], case["top_k"], case["D"], case["F"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that T independent tokens choose, on average
    return {"bytes": int(used * (packed(D, 2 * F) + packed(F, D))) + (E * D + 2 * T * D) * e + 8 * T * k,
            "flops": 6 * T * k * D * F + 2 * T * E * D}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _place(K, device):
    """Byte of its row and shift within it, for the code of each k."""
    k = torch.arange(K, device=device)
    b, w, t, i = k // 128, k % 128 // 32, k % 32 // 8, k % 8
    nib = torch.div(i, 2, rounding_mode="floor") + 4 * (i % 2)
    return 64 * b + 16 * t + 4 * w + nib // 2, 4 * (nib % 2)


def _dense64(wq, sg, zp, K, group):
    byte, shift = _place(K, wq.device)
    w = ((wq[:, byte] >> shift.to(torch.uint8)) & 15).double()
    for g in range(-(-K // group)):
        part = w[:, g * group:(g + 1) * group]
        part -= 8.0 if zp is None else zp[g].double()[:, None]
        part *= sg[g].double()[:, None]
    return w


def _exact_quant(st):
    """The definition's quotients and products are binary32, each correctly rounded; from there on nothing is rounded
    but the scales (bf16) and the values themselves, which are exact in 64 bits."""
    K, group = st["K"], st["group"]

    def r32(a):
        return a.float().double()

    values, scales, zeros = [], [], []
    for k0 in range(0, K, group):
        w = r32(st["W"][k0:k0 + group].double() * st["s"][k0:k0 + group, None].double())
        top, bottom = w.max(0).values, w.min(0).values
        if st["asym"]:
            hi, lo = torch.clamp(top, min=0.0), torch.clamp(bottom, max=0.0)
            sc = r32(r32(hi - lo) / 15.0).float().to(torch.bfloat16).double()
            some = sc > 0
            z = torch.where(some, torch.round(r32(-lo / sc)), torch.zeros_like(sc)).clamp(0, 15)
            q = torch.clamp(torch.round(r32(w / sc)) + z, 0, 15) - z
            zeros.append(z)
        else:
            sc = r32(torch.maximum(top, -bottom) / 7.0).float().to(torch.bfloat16).double()
            some = sc > 0
            q = torch.clamp(torch.round(r32(w / sc)), -7, 7)
        values.append((torch.where(some, q, torch.zeros_like(q)) * sc).T)
        scales.append(sc)
    out = {"values": torch.cat(values, 1), "scales": torch.stack(scales)}
    if st["asym"]:
        out["zeros"] = torch.stack(zeros).to(torch.uint8)
    return out


def _exact_moe(st):
    T, k, D, F, group = st["T"], st["top_k"], st["D"], st["F"], st["group"]
    x = st["x"].double()
    logits = torch.stack([(x * r.double()).sum(-1) for r in st["wr"]], -1)
    e = torch.exp(logits - logits.max(-1, keepdim=True).values)
    p = e / e.sum(-1, keepdim=True)
    left, ids, wts = logits.clone(), [], []
    rows = torch.arange(T, device=x.device)
    for _ in range(k):  # argmax of equal values: the first of them
        best = torch.where(left == left.max(-1, keepdim=True).values, 0, 1).argmin(-1)
        ids.append(best)
        wts.append(p[rows, best])
        left[rows, best] = -math.inf
    ids, wts = torch.stack(ids, -1), torch.stack(wts, -1)
    if st["renorm"]:
        wts = wts / wts.sum(-1, keepdim=True)
    y = torch.zeros(T, D, dtype=torch.float64, device=x.device)
    for ex in ids.unique().tolist():
        t, j = torch.nonzero(ids == ex, as_tuple=True)
        z13, z2 = (None, None) if st["z13"] is None else (st["z13"][ex], st["z2"][ex])
        gu = x[t] @ _dense64(st["w13"][ex], st["s13"][ex], z13, D, group).T
        h = gu[:, :F] / (1.0 + torch.exp(-gu[:, :F])) * gu[:, F:]
        y[t] += wts[t, j, None] * (h @ _dense64(st["w2"][ex], st["s2"][ex], z2, F, group).T)
    return {"y": y, "ids": ids.int(), "weights": wts}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_quant(st)
    if case["op"] == "gemm":
        w = _dense64(st["wq"], st["sg"], st["zp"], st["K"], st["group"])
        return st["x"].double() @ w.T
    return _exact_moe(st)
