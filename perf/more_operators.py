"""Timed cases of the MoE layer's path for many rows (prefill, training).

Five kinds of case, each with a plain form in elementary fp32 torch operations
and the calls of this package's entry points:

* ``gate``     top-k of given router logits with the routing weights, then the
               weights' gradient back to the logits (moe_gate, moe_gate_backward);
* ``tokens``   forward: the picks sorted by expert, the tokens' rows brought into
               that order, and experts' rows brought back as weighted sums
               (moe_sort, moe_dispatch, moe_return); backward: the gradients of
               both (moe_return_backward, moe_return without weights);
* ``mxquant``  rows to MXFP4 (e2m1 values, an e8m0 scale per 32) and read back
               (moe_mx_quant, moe_mx_dequant);
* ``mxproj``   rows times a weight held in MXFP4 (moe_mx_proj: quantise the rows,
               then the product);
* ``mxexperts`` sorted rows times the experts' MXFP4 weights: gate_up with SwiGLU
               from the tokens' rows, or down (moe_mx_gate_up, moe_mx_down).

Sizes follow ``synth.configs``: hidden sizes 4096 and 7168, intermediate 2048,
256 experts of which a GPU holds 32, top-8.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLK = 32  # values an e8m0 scale covers
CHUNK = 128  # columns are padded to whole chunks
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one decode step's rows, the selection steered by a balancing bias
        dict(name="gate_128", op="gate", T=128, E=256, topk=8, score="sigmoid", renorm=1, bias=1),
        # a training batch, softmax probabilities as weights (the gradient reaches every logit)
        dict(name="gate_65536", op="gate", T=65536, E=256, topk=8, score="softmax", renorm=0, bias=0),
        # a decode batch on one of eight GPUs
        dict(name="tokens_64", op="tokens", dir="fwd", T=64, d=4096, E=256, topk=8, n_local=32, base=64, tok="bf16",
             row="bf16"),
        # a prefill chunk on one of eight GPUs, into the fp32 partial that the GPUs add up
        dict(name="tokens_8192", op="tokens", dir="fwd", T=8192, d=7168, E=256, topk=8, n_local=32, base=0, tok="fp32",
             row="bf16"),
        # a training step's backward where one GPU holds every expert
        dict(name="tokens_bwd_4096", op="tokens", dir="bwd", T=4096, d=4096, E=256, topk=8, n_local=256, base=0,
             tok="bf16", row="bf16"),
        # the summed expert partial (fp32) of one decode step
        dict(name="mxquant_8x4096", op="mxquant", M=8, K=4096, x="fp32", back="bf16"),
        # a prefill chunk's hidden rows
        dict(name="mxquant_16384x7168", op="mxquant", M=16384, K=7168, x="bf16", back="bf16"),
        # one token through a gate_up projection
        dict(name="mxproj_1x4096x7168", op="mxproj", M=1, N=4096, K=7168, x="bf16", out="bf16"),
        # ragged in every size (a pruned layer), fp32 result
        dict(name="mxproj_77x4099x2120", op="mxproj", M=77, N=4099, K=2120, x="bf16", out="fp32"),
        # a prefill chunk through a gate_up projection
        dict(name="mxproj_8192x4096x7168", op="mxproj", M=8192, N=4096, K=7168, x="bf16", out="bf16"),
        # uneven popularity in a decode step: buckets from empty to tens of rows
        dict(name="mxdown_64_zipf", op="mxexperts", dir="down", T=64, d=4096, I=2048, E=256, topk=8, n_local=32,
             zipf=1.1, out="bf16"),
        # a prefill chunk through the experts' gate_up
        dict(name="mxgateup_8192", op="mxexperts", dir="gate_up", T=8192, d=4096, I=2048, E=256, topk=8, n_local=32,
             zipf=0.0, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "tokens", "tokens", "mxquant", "mxproj", "mxproj", "mxexperts", "mxexperts"])
    if op == "gate":
        E = rng.choice([8, 60, 100, 128, 255, 256])
        return dict(op=op, T=_log(rng, 1, 65536), E=E, topk=rng.choice([k for k in (1, 2, 6, 8) if k <= E]),
                    score=rng.choice(["sigmoid", "softmax"]), renorm=rng.choice([0, 1]), bias=rng.choice([0, 1]))
    if op == "mxquant":
        return dict(op=op, M=_log(rng, 1, 16384), K=_log(rng, 16, 7168), x=rng.choice(["bf16", "fp32"]),
                    back=rng.choice(["bf16", "fp32"]))
    if op == "mxproj":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 16, 4096), K=_log(rng, 16, 7168),
                    x=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]))
    n_local = rng.choice([1, 3, 8, 31, 32])
    ranks = rng.choice([1, 2, 8])  # as many GPUs share the experts
    E = n_local * ranks
    topk = rng.choice([k for k in (1, 2, 5, 8) if k <= E])
    T = _log(rng, 1, 8192)
    if op == "tokens":
        d = _log(rng, 16, 4096)
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=T, d=d, E=E, topk=topk, n_local=n_local,
                    base=n_local * rng.randrange(ranks), tok=rng.choice(["bf16", "fp32"]),
                    row=rng.choice(["bf16", "fp32"]))
    T = max(1, min(T, 8192 * ranks // topk))
    return dict(op=op, dir=rng.choice(["gate_up", "down"]), T=T, d=128 * _log(rng, 1, 32), I=128 * _log(rng, 1, 16),
                E=E, topk=topk, n_local=n_local, zipf=rng.choice([0.0, 1.1]), out="bf16")


def _padded(K):
    return -(-K // CHUNK) * CHUNK


def work(case):
    c = case
    isz = {"bf16": 2, "fp32": 4}
    if c["op"] == "gate":
        T, E, k = c["T"], c["E"], c["topk"]
        # the gradient looks at every logit only without renormalised softmax weights over the picks
        again = T * E * 4 if c["score"] == "softmax" and not c["renorm"] else T * k * 4
        return {"bytes": T * E * 4 + T * k * 8 + again + T * k * 8 + T * E * 4, "flops": 0}
    if c["op"] == "tokens":
        T, k, d = c["T"], c["topk"], c["d"]
        R = T * k * c["n_local"] / c["E"]  # picks that are local, on average
        tok, row = T * d * isz[c["tok"]], R * d * isz[c["row"]]
        if c["dir"] == "fwd":
            return {"bytes": int(3 * 4 * T * k + 4 * T * k + 2 * (tok + row)), "flops": int(2 * R * d)}
        return {"bytes": int(tok + 2 * row + 12 * T * k + row + tok), "flops": int(4 * R * d)}
    if c["op"] == "mxquant":
        M, K, Kp = c["M"], c["K"], _padded(c["K"])
        q = M * (Kp // 2 + Kp // BLK)
        return {"bytes": M * K * (isz[c["x"]] + isz[c["back"]]) + 2 * q, "flops": 0}
    if c["op"] == "mxproj":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * isz[c["x"]] + N * K * 17 // 32 + M * N * isz[c["out"]], "flops": 2 * M * N * K}
    T, d, I, n = c["T"], c["d"], c["I"], c["n_local"]
    R = T * c["topk"] * n / c["E"]
    active = n * (1.0 - (1.0 - 1.0 / c["E"]) ** (T * c["topk"]))  # evenly popular experts
    if c["dir"] == "gate_up":
        return {"bytes": int(active * 2 * I * d * 17 / 32 + T * d * 2 + R * I * 2), "flops": int(4 * R * d * I)}
    return {"bytes": int(active * d * I * 17 / 32 + R * (I * 17 / 32 + d * 2)), "flops": int(2 * R * d * I)}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(M, K, kind, g):
    """Hidden rows: unit normal, rows of different size, a few large columns."""
    v = torch.randn((M, K), generator=g, device=DEV)
    v *= torch.exp(0.5 * torch.randn((M, 1), generator=g, device=DEV))
    cols = torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)
    v[:, cols] *= 10.0
    return v.to(DTYPES[kind])


def _weights(shape, g):
    """Canonical MXFP4 [..., N, K]: two codes a byte; scales that make a hidden width of 4096 sum to about 1."""
    *lead, N, K = shape
    q = torch.randint(0, 256, (*lead, N, _padded(K) // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(115, 122, (*lead, N, _padded(K) // BLK), generator=g, device=DEV, dtype=torch.uint8)
    return q, s


def _picks(c, g):
    """Distinct picks of T tokens (Gumbel keys, Zipf popularity interleaved over
    the expert ids); the last rows are padding, without a pick."""
    T, E, k = c["T"], c["E"], c["topk"]
    n = c["n_local"]
    e = torch.arange(E, device=DEV)
    rank = (e * max(E // n, 1) + e // n) % E + 1
    u = torch.rand((T, E), generator=g, device=DEV).clamp_(1e-7, 1.0 - 1e-7)
    key = -torch.log(-torch.log(u)) - c.get("zipf", 0.0) * torch.log(rank.float())[None, :]
    ids = torch.topk(key, k, dim=1).indices.to(torch.int32).contiguous()
    pad = T // 50
    if pad:
        ids[T - pad:] = -1
    return ids


def _plain_sort(ids, base, n):
    """counts, offsets, rows, pick_pos: the local picks by expert, then by pick."""
    T, k = ids.shape
    local = (ids >= base) & (ids < base + n)
    key = torch.where(local, ids - base, n).reshape(-1)
    order = torch.sort(key, stable=True).indices
    counts = (key[None, :] == torch.arange(n, device=ids.device)[:, None]).sum(dim=1).to(torch.int32)
    offsets = torch.zeros(n + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(counts, dim=0).to(torch.int32)
    at = torch.arange(T * k, device=ids.device)
    rows = torch.where(at < offsets[n], order // k, -1).to(torch.int32)
    pos = torch.empty_like(at)
    pos[order] = at
    pos = torch.where(local.reshape(-1), pos, -1).to(torch.int32).view(T, k)
    return counts, offsets, rows, pos


def prepare(case, seed):
    c = case
    g = _gen(seed)
    st = dict(case=dict(c))
    mb = None
    if own:
        import moe_decode_layer_router_amd as mb

        st["mb"] = mb
        types = {"bf16": mb.MOE_BF16, "fp32": mb.MOE_FP32}
    op = c["op"]
    if op == "gate":
        T, E, k = c["T"], c["E"], c["topk"]
        # router logits with popular experts; one row in eight holds coarse values (equal logits), one in
        # sixteen has masked experts, and the last rows are padding, masked whole
        st["logits"] = torch.randn((T, E), generator=g, device=DEV) * 1.5 + 0.5 * torch.randn((1, E), generator=g, device=DEV)
        st["logits"][::8] = torch.round(st["logits"][::8] * 4) / 4
        hide = torch.rand((T, E), generator=g, device=DEV) < 0.5
        hide[torch.arange(T, device=DEV) % 16 != 3] = False
        pad = T // 50
        if pad:
            hide[T - pad:] = True
        st["logits"].masked_fill_(hide, -math.inf)
        st["bias"] = 0.3 * torch.randn(E, generator=g, device=DEV) if c["bias"] else None
        st["dw"] = torch.randn((T, k), generator=g, device=DEV)
        st["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        st["w"] = torch.empty((T, k), device=DEV)
        st["dlogits"] = torch.empty((T, E), device=DEV)
        if own:
            st["dims"] = mb.gate_dims_from(dict(
                T=T, E=E, topk=k, renorm=c["renorm"], bias_mode=c["bias"],
                score=mb.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else mb.MOE_SCORE_SOFTMAX))
        return st
    if op == "tokens":
        T, k, d, n = c["T"], c["topk"], c["d"], c["n_local"]
        R = T * k
        tok, row = DTYPES[c["tok"]], DTYPES[c["row"]]
        st["ids"] = _picks(c, g)
        w = torch.rand((T, k), generator=g, device=DEV) + 0.1
        st["w"] = w / w.sum(dim=1, keepdim=True)
        fwd = c["dir"] == "fwd"
        st["x"] = _rows(T, d, c["tok"], g)  # forward: the tokens' rows; backward: the gradient of the sums
        # rows behind the last local pick are not read, and the outputs' are not written: zeros
        st["y"] = torch.zeros((R, d), dtype=row, device=DEV)
        local = int(((st["ids"] >= c["base"]) & (st["ids"] < c["base"] + n)).sum())
        st["n_rows"] = local
        st["y"][:local] = _rows(local, d, c["row"], g) if local else 0
        st["rows_out"] = torch.zeros((R, d), dtype=row, device=DEV)  # dispatched rows, or the gradient of y
        st["tok_out"] = torch.empty((T, d), dtype=tok, device=DEV)  # the weighted sums, or the gradient of x
        st["counts"] = torch.empty(n, dtype=torch.int32, device=DEV)
        st["offsets"] = torch.empty(n + 1, dtype=torch.int32, device=DEV)
        st["rows"] = torch.empty(R, dtype=torch.int32, device=DEV)
        st["pos"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        if not fwd:
            st["counts"], st["offsets"], st["rows"], st["pos"] = _plain_sort(st["ids"], c["base"], n)
            st["dxs"] = torch.zeros((R, d), dtype=row, device=DEV)
            st["dxs"][:local] = _rows(local, d, c["row"], g) if local else 0
            st["dw"] = torch.empty((T, k), device=DEV)
        if own:
            st["dims"] = mb.rows_dims_from(dict(T=T, E=c["E"], topk=k, n_local=n, local_base=c["base"], d=d,
                                                tok_type=types[c["tok"]], row_type=types[c["row"]]))
            st["ws"] = torch.zeros(mb.moe_sort_workspace_bytes(st["dims"]), dtype=torch.uint8, device=DEV)
        return st
    if op in ("mxquant", "mxproj"):
        M, K = c["M"], c["K"]
        st["x"] = _rows(M, K, c["x"], g)
        if M >= 8:
            st["x"][M // 2] = 0  # a padded row
        if op == "mxquant":
            st["q"] = torch.empty((M, _padded(K) // 2), dtype=torch.uint8, device=DEV)
            st["s"] = torch.empty((M, _padded(K) // BLK), dtype=torch.uint8, device=DEV)
            st["out"] = torch.empty((M, K), dtype=DTYPES[c["back"]], device=DEV)
        else:
            st["q"], st["s"] = _weights((c["N"], K), g)
            st["out"] = torch.empty((M, c["N"]), dtype=DTYPES[c["out"]], device=DEV)
        if own:
            st["dims"] = mb.mx_dims_from(dict(M=M, N=c.get("N", 1), K=K, in_type=types[c["x"]],
                                              out_type=types[c["back"] if op == "mxquant" else c["out"]]))
            if op == "mxproj":
                st["packed"] = torch.empty(mb.moe_packed_mx_bytes(st["dims"]), dtype=torch.uint8, device=DEV)
                mb.moe_pack_mx(st["dims"], st["q"], st["s"], st["packed"])
                st["ws"] = torch.zeros(mb.moe_mx_proj_workspace_bytes(st["dims"]), dtype=torch.uint8, device=DEV)
        return st
    T, d, I, n, k = c["T"], c["d"], c["I"], c["n_local"], c["topk"]
    up = c["dir"] == "gate_up"
    counts, st["offsets"], st["rows"], _ = _plain_sort(_picks(c, g), 0, n)
    st["starts"] = st["offsets"].tolist()
    R = T * k
    N, K = (2 * I, d) if up else (d, I)
    st["q"], st["s"] = _weights((n, N, K), g)
    # rows behind the last pick are not written: they stay zero on both sides
    st["out"] = torch.zeros((R, I if up else d), dtype=DTYPES[c["out"]], device=DEV)
    if up:
        st["x"] = _rows(T, d, "bf16", g)
        st["xq"] = torch.empty((T, d // 2), dtype=torch.uint8, device=DEV)
        st["xs"] = torch.empty((T, d // BLK), dtype=torch.uint8, device=DEV)
    else:  # as gate_up's epilogue leaves the rows
        st["xq"] = torch.zeros((R, I // 2), dtype=torch.uint8, device=DEV)
        st["xs"] = torch.zeros((R, I // BLK), dtype=torch.uint8, device=DEV)
        local = st["starts"][-1]
        if local:
            h = torch.nn.functional.silu(_rows(local, I, "fp32", g)) * _rows(local, I, "fp32", g)
            st["xq"][:local], st["xs"][:local] = _plain_codes(h)
    if own:
        st["dims"] = mb.mx_group_dims_from(dict(T=T, E=c["E"], topk=k, n_local=n, d=d, I=I, h_type=mb.MOE_BF16,
                                                out_type=types[c["out"]]))
        if up:
            st["xdims"] = mb.mx_dims_from(dict(M=T, K=d, in_type=mb.MOE_BF16))
        wd = mb.dims_from(dict(S=1, d=d, E=n, topk=1, n_local=n, local_base=0, I=I, renorm=1, eps=1e-6, shared_I=0))
        which = mb.MOE_W13 if up else mb.MOE_W2
        st["packed"] = torch.empty(mb.moe_packed_mxfp4_bytes(wd, which), dtype=torch.uint8, device=DEV)
        mb.moe_pack_mxfp4(wd, which, st["q"], st["s"], st["packed"])
    return st


# ------------------------------------------------------------------ one pass


def run(state):
    st = state
    c = st["case"]
    op = c["op"]
    if own:
        mb = st["mb"]
        d = st["dims"]
        if op == "gate":
            mb.moe_gate(d, st["logits"], st["bias"], st["ids"], st["w"])
            mb.moe_gate_backward(d, st["logits"], st["ids"], st["dw"], None, st["dlogits"])
            return st["ids"], st["w"], st["dlogits"]
        if op == "tokens" and c["dir"] == "fwd":
            mb.moe_sort(d, st["ids"], st["counts"], st["offsets"], st["rows"], st["pos"], st["ws"])
            mb.moe_dispatch(d, st["x"], st["pos"], st["rows_out"])
            mb.moe_return(d, st["y"], st["w"], st["pos"], st["tok_out"])
            return st["counts"], st["offsets"], st["rows"], st["pos"], st["rows_out"], st["tok_out"]
        if op == "tokens":
            mb.moe_return_backward(d, st["x"], st["y"], st["w"], st["pos"], st["rows_out"], st["dw"])
            mb.moe_return(d, st["dxs"], None, st["pos"], st["tok_out"])
            return st["rows_out"], st["dw"], st["tok_out"]
        if op == "mxquant":
            mb.moe_mx_quant(d, st["x"], st["q"], st["s"])
            mb.moe_mx_dequant(d, st["q"], st["s"], st["out"])
            return st["s"], st["out"]
        if op == "mxproj":
            mb.moe_mx_proj(d, st["x"], st["packed"], st["out"], st["ws"])
            return st["out"]
        if c["dir"] == "gate_up":
            mb.moe_mx_quant(st["xdims"], st["x"], st["xq"], st["xs"])
            mb.moe_mx_gate_up(d, st["xq"], st["xs"], st["offsets"], st["rows"], st["packed"], st["out"], None)
        else:
            mb.moe_mx_down(d, st["xq"], st["xs"], st["offsets"], st["packed"], st["out"])
        return st["out"]
    if op == "gate":
        return _plain_gate(st)
    if op == "tokens":
        return _plain_tokens(st)
    if op == "mxquant":
        v, s = _plain_quant(st["x"])
        return s, v[:, :c["K"]].to(st["out"].dtype)
    if op == "mxproj":
        x, _ = _plain_quant(st["x"])
        w = _plain_values(st["q"], st["s"])
        return torch.matmul(x[:, :c["K"]], w[:, :c["K"]].t()).to(st["out"].dtype)
    return _plain_experts(st)


def _plain_gate(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["topk"]
    l = st["logits"]
    left = l + st["bias"][None, :] if c["bias"] else l.clone()
    expert = torch.arange(E, device=DEV)[None, :]
    ids = torch.empty((T, k), dtype=torch.int64, device=DEV)
    for s in range(k):  # the largest key that is left, the lowest expert among equal ones
        top = left.amax(dim=1, keepdim=True)
        e = torch.where(left == top, expert, E).amin(dim=1, keepdim=True)
        ids[:, s:s + 1] = torch.where(top == -math.inf, -1, e)
        left = left.masked_fill(expert == e, -math.inf)
    got = ids >= 0
    at = ids.clamp(min=0)
    v = torch.where(got, l.gather(1, at), -math.inf)  # the picks' logits
    if c["score"] == "sigmoid":
        # sigmoid(l) over a common factor, so that very negative logits keep their ratios
        m = v.amax(dim=1, keepdim=True).clamp(max=0.0) if c["renorm"] else torch.zeros((T, 1), device=DEV)
        m = torch.where(m == -math.inf, 0.0, m)
        a = torch.exp(v.clamp(max=0.0) - m) / (1.0 + torch.exp(-v.abs()))
        slope = 1.0 / (1.0 + torch.exp(v))  # 1 - sigmoid(l)
    else:
        full = v if c["renorm"] else l
        m = full.amax(dim=1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        a = torch.exp(v - m)
        slope = 1.0
    a = torch.where(got, a, 0.0)
    if c["renorm"]:
        total = a.sum(dim=1, keepdim=True)
    elif c["score"] == "softmax":
        total = torch.exp(l - m).sum(dim=1, keepdim=True)
    else:
        total = torch.ones((T, 1), device=DEV)
    w = torch.where(got, a / torch.where(total == 0, 1.0, total), 0.0)
    dw = torch.where(got, st["dw"], 0.0)
    dl = torch.zeros((T, E + 1), device=DEV)
    col = torch.where(got, at, E)
    if c["score"] == "softmax" and not c["renorm"]:
        mean = (dw * w).sum(dim=1, keepdim=True)
        p = torch.exp(l - m) / torch.where(total == 0, 1.0, total)
        dl[:, :E] = -mean * p
        dl.scatter_add_(1, col, dw * w)
    else:
        mean = (dw * w).sum(dim=1, keepdim=True) if c["renorm"] else 0.0
        dl.scatter_(1, col, w * slope * (dw - mean))
    return ids.to(torch.int32), w, dl[:, :E].contiguous()


def _plain_tokens(st):
    c = st["case"]
    T, k, d = c["T"], c["topk"], c["d"]
    tok, row = DTYPES[c["tok"]], DTYPES[c["row"]]
    n = st["n_rows"]
    if c["dir"] == "fwd":
        counts, offsets, rows, pos = _plain_sort(st["ids"], c["base"], c["n_local"])
        xs = torch.zeros((T * k, d), dtype=row, device=DEV)
        xs[:n] = st["x"].float()[rows[:n].long()].to(row)
        src, w = st["y"], st["w"]
    else:
        pos, rows = st["pos"], st["rows"]
        src, w = st["dxs"], None
    out = torch.zeros((T, d), device=DEV)
    for s in range(k):
        p = pos[:, s].long()
        v = src[p.clamp(min=0)].float()
        if w is not None:
            v = v * w[:, s:s + 1]
        out += torch.where((p >= 0)[:, None], v, 0.0)
    if c["dir"] == "fwd":
        return counts, offsets, rows, pos, xs, out.to(tok)
    dy = torch.zeros((T * k, d), dtype=row, device=DEV)
    dw = torch.zeros((T, k), device=DEV)
    g = st["x"].float()
    for s in range(k):
        p = pos[:, s].long()
        on = p >= 0
        dw[:, s] = torch.where(on, (g * st["y"][p.clamp(min=0)].float()).sum(dim=1), 0.0)
        dy[p[on]] = (g * st["w"][:, s:s + 1])[on].to(row)
    return dy, dw, out.to(tok)


def _plain_quant(x):
    """The values that MXFP4 rows stand for (fp32, whole chunks) and the scale bytes."""
    M, K = x.shape
    v = torch.zeros((M, _padded(K)), device=x.device)
    v[:, :K] = x.float()
    v = v.view(M, -1, BLK)
    m, e = torch.frexp(v.abs().amax(dim=2))  # amax = m 2^e, m in [1/2, 1); 7 = 0.875 2^3
    e = torch.where(m < 0.875, e - 3, e - 2).clamp(min=-127)
    e = torch.where(m == 0, -127, e)
    s = torch.where(e == -127, 0x00400000, (e + 127) << 23).to(torch.int32).view(torch.float32)[:, :, None]
    a = (v / s).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.round(a / step) * step  # torch.round: halves to even
    return (torch.where(v < 0, -r, r) * s).view(M, -1), (e + 127).to(torch.uint8)


def _plain_codes(x):
    """MXFP4 bytes of rows (two codes a byte, the even column in the low half) and their scale bytes."""
    v, s = _plain_quant(x)
    M = v.shape[0]
    r = v.view(M, -1, BLK) / _plain_scale(s)[:, :, None]
    a = r.abs().view(M, -1)
    code = torch.zeros(a.shape, dtype=torch.uint8, device=x.device)
    for border in E2M1[1:]:
        code += (a >= border).to(torch.uint8)
    code += 8 * (r.view(M, -1) < 0).to(torch.uint8)
    return code[:, ::2] | (code[:, 1::2] << 4), s


def _plain_scale(s):
    s = s.to(torch.int32)
    return torch.where(s == 0, 0x00400000, s << 23).view(torch.float32)


def _plain_values(q, s):
    """fp32 [..., N, K] of canonical MXFP4 bytes."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=q.device)
    codes = torch.stack((q & 15, q >> 4), dim=-1).to(torch.int32)
    v = table[codes].view(*s.shape, BLK)
    return (v * _plain_scale(s)[..., None]).view(*q.shape[:-1], -1)


def _plain_experts(st):
    c = st["case"]
    up = c["dir"] == "gate_up"
    I = c["I"]
    x = _plain_quant(st["x"])[0] if up else None
    out = torch.zeros_like(st["out"])
    for e in range(c["n_local"]):
        lo, hi = st["starts"][e], st["starts"][e + 1]
        if hi == lo:
            continue
        v = x[st["rows"][lo:hi].long()] if up else _plain_values(st["xq"][lo:hi], st["xs"][lo:hi])
        y = torch.matmul(v, _plain_values(st["q"][e], st["s"][e]).t())
        if up:
            gate = y[:, :I]
            y = gate / (1.0 + torch.exp(-gate)) * y[:, I:]
        out[lo:hi] = y.to(out.dtype)
    return out


# ------------------------------------------------------------------ 64 bits


def _two_to(e):
    """2^e in float64 from its exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_quant(x):
    """float64 values and scale bytes, the scale found by trying exponents in turn."""
    M, K = x.shape
    v = torch.zeros((M, _padded(K)), dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    v = v.view(M, -1, BLK)
    top = v.abs().amax(dim=2)
    _, e = torch.frexp(top)
    e = (e - 5).clamp(min=-127)
    for _ in range(4):
        e = torch.where(top < 7.0 * _two_to(e), e, e + 1)
    e = torch.where(top == 0, -127, e)
    u = (v / _two_to(e)[:, :, None])
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    a = u.abs().contiguous()
    low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # they differ on a tie
    code = torch.where((low != high) & (low % 2 == 1), high, low)
    val = torch.copysign(grid[code], u) * _two_to(e)[:, :, None]
    return val.view(M, -1), (e + 127).to(torch.uint8)


def _exact_values(q, s):
    v = torch.zeros((*q.shape[:-1], q.shape[-1] * 2), dtype=torch.float64, device=q.device)
    for half in (0, 1):
        code = (q >> (4 * half)) & 15
        mag, ex = (code & 1).double(), ((code >> 1) & 3).long()  # 1 mantissa bit, 2 exponent bits, bias 1
        val = torch.where(ex == 0, mag / 2, (1 + mag / 2) * _two_to(ex - 1))
        v[..., half::2] = torch.where(code >= 8, -val, val)
    return (v.view(*s.shape, BLK) * _two_to(s.long() - 127)[..., None]).view(v.shape)


def _exact_gate(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["topk"]
    l = st["logits"].double()
    key = (st["logits"] + st["bias"][None, :]) if c["bias"] else st["logits"]  # the key is an fp32 sum
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids = torch.where(order.values[:, :k] == -math.inf, -1, order.indices[:, :k])
    pick = torch.nn.functional.one_hot(ids.clamp(min=0), E).bool() & (ids >= 0)[:, :, None]  # [T, k, E]
    on = pick.any(dim=1)
    if c["score"] == "sigmoid":
        logp = torch.nn.functional.logsigmoid(l)
        if c["renorm"]:
            logp = torch.log_softmax(logp.masked_fill(~on, -math.inf), dim=1)
    else:
        logp = torch.log_softmax(l.masked_fill(~on, -math.inf) if c["renorm"] else l, dim=1)
    p = torch.nan_to_num(torch.exp(logp), nan=0.0)  # a row without a logit: zeros
    w = torch.where(pick, p[:, None, :], 0.0).sum(dim=2)
    G = torch.where(pick, st["dw"].double()[:, :, None], 0.0).sum(dim=1)
    mean = (G * torch.where(on, p, 0.0)).sum(dim=1, keepdim=True)
    if c["score"] == "sigmoid":
        dl = torch.where(on, p * torch.sigmoid(-l) * (G - (mean if c["renorm"] else 0.0)), 0.0)
    else:
        dl = p * (G - mean)
        if c["renorm"]:
            dl = torch.where(on, dl, 0.0)
    return ids.to(torch.int32), w, dl


def _exact_tokens(st):
    c = st["case"]
    T, k, d, n, base = c["T"], c["topk"], c["d"], c["n_local"], c["base"]
    ids = st["ids"].cpu().numpy()
    flat = ids.reshape(-1)
    lists = [np.nonzero(flat == base + e)[0] for e in range(n)]
    counts = np.array([len(p) for p in lists], np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    order = np.concatenate(lists)
    rows = np.full(T * k, -1, np.int32)
    rows[:len(order)] = order // k
    pos = np.full(T * k, -1, np.int32)
    pos[order] = np.arange(len(order))
    order = torch.from_numpy(order).to(DEV)
    t = order // k
    m = len(order)
    w = st["w"].double().reshape(-1)[order][:, None]
    x = st["x"]
    big = torch.zeros((T * k, d), dtype=torch.float64, device=DEV)
    out = torch.zeros((T, d), dtype=torch.float64, device=DEV)
    if c["dir"] == "fwd":
        big[:m] = x.double()[t]
        out.index_add_(0, t, st["y"][:m].double() * w)
        as_t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
        return as_t(counts), as_t(offsets), as_t(rows), as_t(pos).view(T, k), big, out
    big[:m] = x.double()[t] * w
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[order] = (x.double()[t] * st["y"][:m].double()).sum(dim=1)
    out.index_add_(0, t, st["dxs"][:m].double())
    return big, dw.view(T, k), out


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    op = c["op"]
    if op == "gate":
        return _exact_gate(st)
    if op == "tokens":
        return _exact_tokens(st)
    if op == "mxquant":
        v, s = _exact_quant(st["x"])
        return s, v[:, :c["K"]].contiguous()
    if op == "mxproj":
        x, _ = _exact_quant(st["x"])
        w = _exact_values(st["q"], st["s"])
        return torch.matmul(x[:, :c["K"]].contiguous(), w[:, :c["K"]].t().contiguous())
    up = c["dir"] == "gate_up"
    x = _exact_quant(st["x"])[0] if up else _exact_values(st["xq"], st["xs"])
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for e in range(c["n_local"]):
        r = slice(st["starts"][e], st["starts"][e + 1])
        if r.start == r.stop:
            continue
        v = x[st["rows"][r].long()] if up else x[r]
        y = torch.matmul(v, _exact_values(st["q"][e], st["s"][e]).t().contiguous())
        if up:
            y = y[:, :c["I"]] * torch.sigmoid(y[:, :c["I"]]) * y[:, c["I"]:]
        out[r] = y
    return out
