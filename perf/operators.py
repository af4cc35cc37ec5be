"""What is measured of the linear, grouped and SwiGLU operators.

Three operators, each in every direction a user calls it:

- "linear" / "linear_dx": rows times an affine-packed matrix (4 or 8 bits, a bf16 scale and bias per
  group along the input) and the gradient of its input through the frozen packed weights;
- "grouped": rows sorted by expert times each expert's own matrix (forward, input gradient, weight
  gradient), group sizes known to the device as offsets, the rows behind the last group left alone;
- "swiglu": w * silu(gate) * up on stacked [gate | up] rows with a weight per row, and its gradient.

With `own` false `run` computes them in plain torch operations in 32 bits; with `own` true it calls
the library.
"""
import math

import torch

own = False

BF16, F16, F32 = 0, 1, 2  # the library's type codes
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE = {"bf16": BF16, "fp16": F16, "fp32": F32}


def listed():
    return [
        # one token through a projection of the 2048-wide layer (its expert width, 512): the smallest
        # call of decoding, all latency
        {"name": "linear_decode", "op": "linear", "T": 1, "K": 2048, "N": 512, "bits": 4, "group": 64},
        # one token against a vocabulary-sized output: the largest matrix-vector product, all bandwidth
        {"name": "linear_head", "op": "linear", "T": 1, "K": 2048, "N": 131072, "bits": 4, "group": 64},
        # eight decoding requests through a square projection, packed at group 32
        {"name": "linear_batch8_g32", "op": "linear", "T": 8, "K": 2048, "N": 2048, "bits": 4, "group": 32},
        # an odd batch through an 8-bit layer of odd sizes (a gate or a head that is kept at 8 bits)
        {"name": "linear_odd_int8", "op": "linear", "T": 13, "K": 1056, "N": 1003, "bits": 8, "group": 32},
        # a 2048-token prompt through a packed projection
        {"name": "linear_prefill", "op": "linear", "T": 2048, "K": 2048, "N": 4096, "bits": 4, "group": 64},
        # the gradient of that projection's input: adapter training over the frozen packed base
        {"name": "linear_dx", "op": "linear_dx", "T": 2048, "K": 2048, "N": 4096, "bits": 4, "group": 64},
        # eight tokens at top-4 on 256 unquantised experts: one row or none per expert, gate|up rows
        {"name": "grouped_decode", "op": "grouped", "dir": "fwd", "M": 34, "G": 256, "N": 1024, "K": 2048,
         "dtype": "bf16", "skew": 0.5},
        # a 2048-token prompt at top-8: about 64 rows per expert, ragged
        {"name": "grouped_prefill", "op": "grouped", "dir": "fwd", "M": 17472, "G": 256, "N": 1024, "K": 2048,
         "dtype": "bf16", "skew": 0.8},
        # training on fewer, larger experts: the gradient of the rows, in fp16
        {"name": "grouped_dx", "op": "grouped", "dir": "dx", "M": 16384, "G": 16, "N": 1024, "K": 2048,
         "dtype": "fp16", "skew": 0.5},
        # and of the experts' weights, kept in fp32 as optimizers take it
        {"name": "grouped_dw", "op": "grouped", "dir": "dw", "M": 16384, "G": 64, "N": 1024, "K": 2048,
         "dtype": "bf16", "out": "fp32", "skew": 0.5},
        # the activation between the two products of the prompt's experts
        {"name": "swiglu_prefill", "op": "swiglu", "dir": "fwd", "M": 17472, "I": 512, "dtype": "bf16"},
        # its gradient in training
        {"name": "swiglu_dx", "op": "swiglu", "dir": "dx", "M": 16384, "I": 1024, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_dx", "grouped", "grouped", "grouped", "swiglu"])
    if kind in ("linear", "linear_dx"):
        bits, group = rng.choice([4, 4, 8]), rng.choice([32, 64, 64, 128])
        T = _log(rng, 1, 2048)
        K = group * max(1, _log(rng, 64, 8192) // group)
        most = min(131072, (1 << 28) // K, (1 << 34) // (K * T))
        N = _log(rng, 16, max(17, most)) if rng.random() < 0.5 else 8 * max(2, _log(rng, 16, max(17, most)) // 8)
        return {"op": kind, "T": T, "K": K, "N": N, "bits": bits, "group": group}
    if kind == "grouped":
        d = rng.choice(["fwd", "dx", "dw"])
        M, G = _log(rng, 1, 16384), _log(rng, 1, 256)
        odd = rng.random() < 0.25
        N, K = _log(rng, 16, 2048), _log(rng, 16, 2048)
        if not odd:
            N, K = 8 * max(2, N // 8), 8 * max(2, K // 8)
        case = {"op": "grouped", "dir": d, "M": M, "G": G, "N": N, "K": K, "dtype": rng.choice(["bf16", "fp16"]),
                "skew": round(rng.uniform(0.0, 0.8), 2)}
        if d == "dw":
            case["out"] = rng.choice([case["dtype"], "fp32"])
        return case
    return {"op": "swiglu", "dir": rng.choice(["fwd", "dx"]), "M": _log(rng, 1, 16384), "I": _log(rng, 16, 1024),
            "dtype": rng.choice(["bf16", "fp16"])}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _packed(g, N, K, bits, group):
    """Weights N(0, 0.02) in the packed format: group minimum as the bias, a bf16 scale that covers
    the range, codes low field first in 32-bit words."""
    words = torch.empty((N, K * bits // 32), dtype=torch.int32, device="cuda")
    scales = torch.empty((N, K // group), dtype=torch.bfloat16, device="cuda")
    biases = torch.empty_like(scales)
    shift = torch.arange(0, 32, bits, device="cuda")
    for n in range(0, N, 32768):  # bounds the 32-bit intermediates
        w = _normal(g, (min(32768, N - n), K // group, group), 0.02)
        lo, hi = w.amin(2), w.amax(2)
        b = lo.to(torch.bfloat16)
        s = ((hi - b.float()) / (2 ** bits - 1)).to(torch.bfloat16)
        q = ((w - b.float()[..., None]) / s.float()[..., None]).round().clamp(0, 2 ** bits - 1)
        q = q.to(torch.int64).view(w.shape[0], -1, 32 // bits)
        u = (q << shift).sum(2)
        words[n:n + len(w)] = torch.where(u >= 1 << 31, u - (1 << 32), u).to(torch.int32)
        scales[n:n + len(w)], biases[n:n + len(w)] = s, b
    return words, scales, biases


def _sizes(case, seed):
    """Rows of each group: skewed shares, some groups empty, about one row in sixteen behind the last."""
    c = torch.Generator().manual_seed(int(seed) * 7919 + 13)
    M, G = case["M"], case["G"]
    share = torch.exp(case["skew"] * torch.randn(G, generator=c)) * (torch.rand(G, generator=c) > 0.06)
    if not share.sum() > 0:
        share[0] = 1.0
    used = M - M // 16
    return torch.bincount(torch.multinomial(share, used, replacement=True, generator=c), minlength=G)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op in ("linear", "linear_dx"):
        T, K, N = case["T"], case["K"], case["N"]
        s["words"], s["scales"], s["biases"] = _packed(g, N, K, case["bits"], case["group"])
        a, b = (K, N) if op == "linear" else (N, K)
        s["x"] = _normal(g, (T, a), 1.0, torch.bfloat16)
        s["y"] = torch.zeros((T, b), dtype=torch.bfloat16, device="cuda")
        if own:  # the descriptor and the scratch that a program keeps next to its weights
            import int4_group_affine_b200 as m
            q = m.QTensor()
            q.packed, q.scales, q.biases = s["words"].data_ptr(), s["scales"].data_ptr(), s["biases"].data_ptr()
            q.n, q.out, q.in_, q.bits, q.group = 1, N, K, case["bits"], case["group"]
            size = m.moe_affine_linear_workspace_bytes if op == "linear" else m.moe_affine_linear_dx_workspace_bytes
            s["q"], s["bytes"] = q, size(q, T)
            s["ws"] = torch.empty(s["bytes"], dtype=torch.uint8, device="cuda")
            m.moe_workspace_init(s["ws"], s["bytes"])
        return s
    dtype = TORCH[case["dtype"]]
    if op == "grouped":
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        n = _sizes(case, seed)
        s["most"] = int(n.max())
        s["off"] = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).cuda()
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if case["dir"] != "dw":
            s["W"] = torch.empty((G, N, K), dtype=dtype, device="cuda")
            for e in range(0, G, 32):
                s["W"][e:e + 32] = _normal(g, (min(32, G - e), N, K), 0.02, dtype)
        if case["dir"] != "dx":
            s["x"] = _normal(g, (M, K), 1.0, dtype)
        if case["dir"] != "fwd":
            s["dy"] = _normal(g, (M, N), 1.0, dtype)
        shape = {"fwd": (M, N), "dx": (M, K), "dw": (G, N, K)}[case["dir"]]
        s["out"] = torch.zeros(shape, dtype=TORCH[case["out"]] if case["dir"] == "dw" else dtype, device="cuda")
        return s
    M, I = case["M"], case["I"]
    s["rows"] = torch.tensor([0, M - M // 16], dtype=torch.int32, device="cuda")
    s["gu"] = _normal(g, (M, 2 * I), 1.5, dtype)
    s["w"] = torch.rand(M, generator=g, device="cuda")
    if case["dir"] == "fwd":
        s["h"] = torch.zeros((M, I), dtype=dtype, device="cuda")
    else:
        s["dh"] = _normal(g, (M, I), 1.0, dtype)
        s["dgu"] = torch.zeros((M, 2 * I), dtype=dtype, device="cuda")
        s["dw"] = torch.zeros(M, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _weights(s):
    """The packed matrix in 32 bits: each code times its group's scale, plus its bias."""
    c = s["case"]
    shift = torch.arange(0, 32, c["bits"], device="cuda", dtype=torch.int32)
    q = (s["words"][..., None] >> shift) & (2 ** c["bits"] - 1)
    q = q.view(c["N"], c["K"] // c["group"], c["group"]).float()
    return (q * s["scales"].float()[..., None] + s["biases"].float()[..., None]).view(c["N"], c["K"])


def _plain_linear(s):
    w, x = _weights(s), s["x"].float()
    return (x @ w.t() if s["case"]["op"] == "linear" else x @ w).to(torch.bfloat16)


def _plain_grouped(s):
    c = s["case"]
    M, G, R = c["M"], c["G"], s["most"]
    off = s["off"].long()
    row = torch.arange(M, device="cuda")
    grp = torch.searchsorted(off[1:].contiguous(), row, right=True)  # G for the rows behind the last group
    pos = (row - off[grp]) % max(R, 1)
    valid = (grp < G)[:, None]

    def by_group(v):
        out = torch.zeros((G + 1, R, v.shape[1]), device="cuda")
        out[grp, pos] = v.float()
        return out[:G]

    def by_row(v):
        return torch.where(valid, v[grp.clamp(max=G - 1), pos], 0.0).to(TORCH[c["dtype"]])

    if c["dir"] == "fwd":
        return by_row(by_group(s["x"]) @ s["W"].float().transpose(1, 2))
    if c["dir"] == "dx":
        return by_row(by_group(s["dy"]) @ s["W"].float())
    return (by_group(s["dy"]).transpose(1, 2) @ by_group(s["x"])).to(TORCH[c["out"]])


def _plain_swiglu(s):
    c = s["case"]
    dtype, I = TORCH[c["dtype"]], c["I"]
    valid = (torch.arange(c["M"], device="cuda") < s["rows"][1])[:, None]
    gate, up, w = s["gu"][:, :I].float(), s["gu"][:, I:].float(), s["w"][:, None]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    if c["dir"] == "fwd":
        return torch.where(valid, w * gate * sig * up, 0.0).to(dtype)
    dh = s["dh"].float()
    dgate = w * dh * up * sig * (1.0 + gate * (1.0 - sig))
    dup = w * dh * gate * sig
    dw = (dh * gate * sig * up).sum(1)
    return [torch.where(valid, torch.cat([dgate, dup], 1), 0.0).to(dtype), torch.where(valid[:, 0], dw, 0.0)]


# ------------------------------------------------------------------ a pass


def _own(s):
    import int4_group_affine_b200 as m
    c = s["case"]
    if c["op"] == "linear":
        m.moe_affine_linear(s["q"], s["x"], c["T"], s["y"], s["ws"], s["bytes"])
        return s["y"]
    if c["op"] == "linear_dx":
        m.moe_affine_linear_dx(s["q"], s["x"], c["T"], s["y"], s["ws"], s["bytes"])
        return s["y"]
    if c["op"] == "grouped":
        size, code, out, st = (c["M"], c["G"], c["N"], c["K"]), CODE[c["dtype"]], s["out"], s["status"]
        if c["dir"] == "fwd":
            m.moe_grouped_matmul(code, s["x"], s["off"], s["W"], *size, out, st)
        elif c["dir"] == "dx":
            m.moe_grouped_matmul_dx(code, s["dy"], s["off"], s["W"], *size, out, st)
        else:
            m.moe_grouped_matmul_dw(code, s["dy"], s["x"], s["off"], *size, CODE[c["out"]], 0, out, st)
        return out
    if c["dir"] == "fwd":
        m.moe_swiglu(CODE[c["dtype"]], s["gu"], s["w"], s["rows"], 1, c["M"], c["I"], s["h"])
        return s["h"]
    m.moe_swiglu_grad(CODE[c["dtype"]], s["gu"], s["w"], s["dh"], s["rows"], 1, c["M"], c["I"], s["dgu"], s["dw"])
    return [s["dgu"], s["dw"]]


def run(state):
    if own:
        return _own(state)
    return {"l": _plain_linear, "g": _plain_grouped, "s": _plain_swiglu}[state["case"]["op"][0]](state)


def work(case):
    c = case
    if c["op"] in ("linear", "linear_dx"):
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": N * K * c["bits"] // 8 + 4 * N * K // c["group"] + 2 * T * (K + N), "flops": 2 * T * K * N}
    if c["op"] == "grouped":
        used, G, N, K = c["M"] - c["M"] // 16, c["G"], c["N"], c["K"]
        rows = 2 * used * (N + K)
        if c["dir"] == "dw":
            return {"bytes": rows + G * N * K * (4 if c["out"] == "fp32" else 2), "flops": 2 * used * N * K}
        # the matrices of the groups that have rows; about that many when there are few rows
        live = G * (1.0 - (1.0 - 1.0 / G) ** used) if G > 1 else 1
        return {"bytes": rows + 2 * int(live) * N * K, "flops": 2 * used * N * K}
    used, I = c["M"] - c["M"] // 16, c["I"]
    return {"bytes": used * (I * (6 if c["dir"] == "fwd" else 10) + (4 if c["dir"] == "fwd" else 8)),
            "flops": used * I * (6 if c["dir"] == "fwd" else 14)}


# ------------------------------------------------------------------ the definition, in 64 bits


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("linear", "linear_dx"):
        N, K = c["N"], c["K"]
        fields = s["words"].view(torch.uint8)  # little-endian bytes: the lower fields first
        if c["bits"] == 4:
            fields = torch.stack([fields % 16, fields // 16], 2)
        rep = lambda v: v.double().repeat_interleave(c["group"], 1)  # noqa: E731
        x, outs = s["x"].double(), []
        for n in range(0, N, 16384):
            w = fields[n:n + 16384].reshape(-1, K).double() * rep(s["scales"][n:n + 16384]) + rep(s["biases"][n:n + 16384])
            outs.append(torch.einsum("tk,nk->tn", x, w) if c["op"] == "linear"
                        else torch.einsum("tn,nk->tk", x[:, n:n + 16384], w))
        return torch.cat(outs, 1) if c["op"] == "linear" else sum(outs)
    if c["op"] == "grouped":
        off, out = s["off"].tolist(), torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(c["G"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            if c["dir"] == "fwd":
                out[a:b] = torch.einsum("mk,nk->mn", s["x"][a:b].double(), s["W"][e].double())
            elif c["dir"] == "dx":
                out[a:b] = torch.einsum("mn,nk->mk", s["dy"][a:b].double(), s["W"][e].double())
            else:
                out[e] = torch.einsum("mn,mk->nk", s["dy"][a:b].double(), s["x"][a:b].double())
        return out
    used, I = int(s["rows"][1]), c["I"]
    gate, up = s["gu"].double().split(I, 1)
    w, silu = s["w"].double()[:, None], gate * torch.sigmoid(gate)
    if c["dir"] == "fwd":
        h = w * silu * up
        h[used:] = 0
        return h
    dh = s["dh"].double()
    slope = torch.sigmoid(gate) + silu * torch.sigmoid(-gate)
    dgu = torch.cat([w * dh * up * slope, w * dh * silu], 1)
    dw = torch.einsum("mi,mi->m", dh, silu * up)
    dgu[used:], dw[used:] = 0, 0
    return [dgu, dw]
