"""Cases and plain forms of the operators between the MoE layer and the rest of
a model: routing by scores and its gradient, the root-mean-square norm with the
residual's addition and its gradient, and clipping by the global gradient norm.

`run` computes a case with elementary torch operations, or, with `own` set,
with the calls a user makes of the package. `exact` computes the same outputs
in fp64 from the definitions.

Routing of a token with logits l (b: bias of the choice, or 0):
    s_e = softmax(l)_e or 1 / (1 + exp(-l_e))        c_e = s_e + b_e
the top_groups groups whose group_top highest c have the highest sum, in them
the k experts of the highest c (ties: the lower index), with the weights
    w_j = scale * s_j, or scale * s_j / (sum of the kept s)
Padding rows choose nothing (ids -1, weights 0). Then each expert's rows, padded
to the block size. Backwards: the logits' gradient from the weights'.
Norm: h = x + residual, y = w * h / sqrt(mean(h^2) + eps); in 8 bits e4m3 values
of y / s with s = max |y| / 448 of a row or of a group of columns. Backwards
(n = h / sqrt(mean(h^2) + eps), r = 1 / sqrt(...)):
    dh = dresidual + r * (w dy - n * mean(w dy n))        dw = sum over the rows of dy n
Clipping: all gradients times max_norm / norm where norm = sqrt(sum of all squares) is larger.
"""
import math
import random

import numpy as np
import torch

own = False

HIDDEN, INTER, EXPERTS = 7168, 2048, 384  # the 384-expert layer of the package's workloads
EPS = 1e-6
E4M3_MAX = 448.0
TINY = 2.0 ** -126


def _route(name, M, E, k, scoring, bias=False, groups=(1, 1, 1), renorm=True, scale=1.0, masked=False, coarse=False,
           block=0):
    return {"name": name, "op": "route", "M": M, "E": E, "k": k, "scoring": scoring, "bias": bias, "G": groups[0],
            "top_groups": groups[1], "group_top": groups[2], "renorm": renorm, "scale": scale, "masked": masked,
            "coarse": coarse, "block": block}


def _route_bwd(name, M, E, k, scoring, renorm, scale, base, masked):
    return {"name": name, "op": "route_bwd", "M": M, "E": E, "k": k, "scoring": scoring, "renorm": renorm,
            "scale": scale, "base": base, "masked": masked}


def _norm(name, M, N, stream, out=True, quant=0, keep=False, gap=0):
    """stream: type of the residual stream ("none": x alone); quant: columns that share a scale (0: no 8-bit output)."""
    return {"name": name, "op": "norm", "M": M, "N": N, "stream": stream, "out": out, "quant": quant, "keep": keep,
            "gap": gap}


def _norm_bwd(name, M, N, stream, passed):
    return {"name": name, "op": "norm_bwd", "M": M, "N": N, "stream": stream, "passed": passed}


def _clip(name, layers, L, r, K, N, half, ratio):
    """Gradients of the adapters of some layers; ratio: max_norm over their norm."""
    return {"name": name, "op": "clip", "layers": layers, "L": L, "r": r, "K": K, "N": N, "half": half, "ratio": ratio}


def listed():
    return [
        # one stream decoding: latency of routing and grouping
        _route("route_one_token", 1, EXPERTS, 8, "sigmoid", bias=True, scale=2.5, block=16),
        # prompts of a batch with padding, experts in groups
        _route("route_prompts", 4096, 256, 8, "sigmoid", bias=True, groups=(8, 4, 2), scale=2.5, masked=True, block=32),
        # a training batch: softmax over all experts, logits of a bf16 projection (equal ones are common)
        _route("route_batch", 16384, EXPERTS, 8, "softmax", renorm=False, coarse=True),
        # its backward pass
        _route_bwd("route_bwd_batch", 16384, EXPERTS, 8, "softmax", False, 1.0, False, False),
        # sigmoid weights, an odd batch of few experts, added to the balance loss's gradient
        _route_bwd("route_bwd_odd", 4099, 60, 4, "sigmoid", True, 2.5, True, True),
        # one stream decoding
        _norm("norm_one_token", 1, HIDDEN, "bf16"),
        # prompts, for experts on other devices: 8 bits to send beside the router's bf16, fp32 stream
        _norm("norm_prompts_8bit", 2048, HIDDEN, "f32", quant=128),
        # a training batch
        _norm("norm_batch", 16384, HIDDEN, "bf16", keep=True),
        # its backward pass
        _norm_bwd("norm_bwd_batch", 16384, HIDDEN, "bf16", True),
        # a narrow odd batch, fp32 stream
        _norm_bwd("norm_bwd_odd", 1999, 1000, "f32", True),
        # the router's adapters
        _clip("clip_router", 1, 4, 8, HIDDEN, EXPERTS, False, 0.3),
        # the adapters of many layers
        _clip("clip_layers", 24, 8, 64, HIDDEN, HIDDEN, False, 0.3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    kind = rng.random()
    if kind < 0.5:
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, EXPERTS, 512, rng.randint(9, 1024), 1024])
        M = _log(rng, 1, min(16384, 16384 * EXPERTS // E))
        scoring = rng.choice(["softmax", "sigmoid"])
        renorm, scale = rng.random() < 0.6, rng.choice([1.0, 2.5])
        if kind < 0.2:
            case = _route_bwd("", M, E, rng.randint(1, min(8, E)), scoring, renorm, scale, rng.random() < 0.5,
                              rng.random() < 0.5)
        else:
            G = rng.choice([g for g in range(1, 33) if E % g == 0])
            top = rng.randint(1, G)
            k = rng.randint(1, min(8, top * (E // G)))
            case = _route("", M, E, k, scoring, rng.random() < 0.6, (G, top, rng.randint(1, min(2, E // G))), renorm,
                          scale, rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 16, 32, 64]))
    elif kind < 0.85:
        N = rng.choice([512, 1024, INTER, 4096, HIDDEN, 128 * rng.randint(1, 128), 8 * rng.randint(1, 1024),
                        rng.randint(17, 9000)])
        M = _log(rng, 1, min(16384, 16384 * HIDDEN // N // 2))
        if kind < 0.7:
            quant = rng.choice([0, 0, N] + [q for q in (32, 64, 128) if N % q == 0])
            case = _norm("", M, N, rng.choice(["none", "bf16", "bf16", "f32"]), quant == 0 or rng.random() < 0.5, quant,
                         rng.random() < 0.5, rng.choice([0, 0, 8, 24, 5]))
        else:
            case = _norm_bwd("", M, N, rng.choice(["none", "bf16", "f32"]), rng.random() < 0.7)
            if case["stream"] == "none":
                case["passed"] = False
    else:
        r = rng.choice([8, 16, 24, 32, 64])
        K = rng.choice([512, 1024, INTER, 4096, HIDDEN, 8 * rng.randint(16, 896)])
        N = rng.choice([60, 129, EXPERTS, 1000, INTER, HIDDEN])
        case = _clip("", _log(rng, 1, 24), _log(rng, 1, 8), r, K, N, rng.random() < 0.4, rng.choice([0.01, 0.3, 1.7]))
    del case["name"]
    return case


def work(case):
    op = case["op"]
    if op == "route":
        M, E, k = case["M"], case["E"], case["k"]
        grouped = 4.0 * M * k + 4 * (E + 1) if case["block"] else 0.0
        return {"bytes": 4.0 * M * E + 4 * E * case["bias"] + M * case["masked"] + 8.0 * M * k + grouped,
                "flops": 5.0 * M * E}
    if op == "route_bwd":
        M, E, k = case["M"], case["E"], case["k"]
        full = case["scoring"] == "softmax" and not case["renorm"]
        return {"bytes": 4.0 * M * E * (1 + case["base"]) + 4.0 * M * (E if full else k) + 8.0 * M * k,
                "flops": 6.0 * M * (E if full else k) + M * E}
    if op == "norm":
        M, N = case["M"], case["N"]
        s = {"none": 0, "bf16": 2, "f32": 4}[case["stream"]]
        q = 1.0 * M * N + 4.0 * M * (N // case["quant"]) if case["quant"] else 0.0
        return {"bytes": (2.0 + 2 * s + 2 * case["out"]) * M * N + q + 2 * N + 4 * M * case["keep"], "flops": 5.0 * M * N}
    if op == "norm_bwd":
        M, N = case["M"], case["N"]
        s = 4 if case["stream"] == "f32" else 2
        return {"bytes": (2.0 + 2 * s + s * case["passed"]) * M * N + 4 * M + 6 * N, "flops": 9.0 * M * N}
    n = float(case["layers"]) * case["L"] * case["r"] * (case["K"] + case["N"])
    return {"bytes": n * (4 if case["half"] else 8), "flops": 3 * n}


def _logits(case, g):
    M, E = case["M"], case["E"]
    logits = torch.randn(M, E, generator=g, device="cuda") + 0.7 * torch.randn(1, E, generator=g, device="cuda")
    return logits.to(torch.bfloat16).float() if case.get("coarse") else logits


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)

    op, st = case["op"], {"case": case}
    if op in ("route", "route_bwd"):
        M, E, k = case["M"], case["E"], case["k"]
        st["logits"] = _logits(case, g)
        valid = torch.rand(M, generator=g, device="cuda") > 0.1 if case["masked"] else None
        if op == "route":
            st["bias"] = normal(E, scale=0.05) if case["bias"] else None
            st["valid"] = valid
            if valid is not None:  # padding rows hold whatever was left there
                st["logits"][~valid] = float("nan")
            return st
        ids = st["logits"].topk(k, dim=1).indices.to(torch.int32)
        st["ids"] = (ids if valid is None else torch.where(valid[:, None], ids, -1)).contiguous()
        st["dweights"] = normal(M, k, scale=0.01)
        st["base"] = normal(M, E, scale=1e-3) if case["base"] else None
        return st
    if op in ("norm", "norm_bwd"):
        M, N = case["M"], case["N"]
        dtype = torch.float32 if case["stream"] == "f32" else torch.bfloat16
        st["w"] = (1.0 + 0.2 * normal(N)).to(torch.bfloat16)
        loud = torch.where(torch.rand(N, generator=g, device="cuda") < 0.01, 20.0, 1.0)  # a few channels are large
        if op == "norm":
            st["x"] = normal(M, N + case["gap"], dtype=torch.bfloat16)[:, :N]
            st["res"] = None if case["stream"] == "none" else (3 * normal(M, N) * loud).to(dtype)
            return st
        st["h"] = (3 * normal(M, N) * loud).to(dtype)
        st["r"] = 1 / torch.sqrt((st["h"].float() ** 2).mean(1) + EPS)
        st["dy"] = normal(M, N, scale=0.02, dtype=torch.bfloat16)
        st["dres"] = normal(M, N, scale=0.02, dtype=dtype) if case["passed"] else None
        return st
    L, r, K, N = (case[n] for n in ("L", "r", "K", "N"))
    dtype = torch.bfloat16 if case["half"] else torch.float32
    st["grads"] = [normal(*shape, scale=0.01, dtype=dtype) for _ in range(case["layers"])
                   for shape in ((L, r, K), (L, N, r))]
    n = sum(t.numel() for t in st["grads"])
    st["max_norm"] = case["ratio"] * 0.01 * math.sqrt(n)
    return st


# ------------------------------------------------------------------ plain forms
def _scores(scoring, logits):
    """Scores in fp64: the choice compares values that lie close together."""
    l = logits.double()
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _highest(v, n):
    """Places of the n highest values of each row, the highest first, equal ones in order."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


def _plain_route(st):
    c = st["case"]
    M, E, k, G = c["M"], c["E"], c["k"], c["G"]
    live = torch.ones(M, dtype=torch.bool, device="cuda") if st["valid"] is None else st["valid"]
    logits = torch.where(live[:, None], st["logits"], 0.0)
    s = _scores(c["scoring"], logits)
    biased = s + st["bias"].double() if st["bias"] is not None else s
    key = biased if st["bias"] is not None else logits.double()
    if c["top_groups"] < G:
        best = torch.sort(biased.view(M, G, E // G), dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
        chosen = torch.zeros(M, G, dtype=torch.bool, device="cuda").scatter_(1, _highest(best, c["top_groups"]), True)
        key = torch.where(chosen.repeat_interleave(E // G, dim=1), key, -math.inf)
    ids = _highest(key, k)
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    out = {"ids": torch.where(live[:, None], ids, -1).to(torch.int32),
           "weights": (c["scale"] * w * live[:, None]).float()}
    if c["block"]:
        out.update(_plain_grouping(out["ids"], E, c["block"]))
    return out


def _plain_grouping(ids, E, block):
    n = ids.numel()
    flat = torch.where(ids >= 0, ids, E).reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))
    padded = (counts[:E] + block - 1) // block * block
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), padded.cumsum(0)])
    before = counts.cumsum(0) - counts
    expert = flat[order]
    cap = (n + min(E, n) * (block - 1) + block - 1) // block * block
    place = offsets[expert] + torch.arange(n, device="cuda") - before[expert]
    # assignments of no expert go to a place behind the end
    place = torch.where(expert < E, place, cap)
    rows = torch.full((cap + 1,), n, dtype=torch.int32, device="cuda")
    rows[place] = torch.where(expert < E, order, n).to(torch.int32)
    starts = torch.arange(0, cap, block, device="cuda")
    of_block = torch.searchsorted(offsets[1:].contiguous(), starts, right=True)
    of_block = torch.where(starts < offsets[E], of_block, -1)
    return {"rows": rows[:cap], "blocks": of_block.to(torch.int32), "offsets": offsets.to(torch.int32),
            "npp": offsets[E:].to(torch.int32)}


def _plain_route_bwd(st):
    c = st["case"]
    M, E = c["M"], c["E"]
    has = st["ids"] >= 0
    ids = st["ids"].clamp(min=0).long()
    g = torch.where(has, st["dweights"] * c["scale"], 0.0)
    l = st["logits"].gather(1, ids)
    if c["scoring"] == "softmax" and not c["renorm"]:
        e = torch.exp(st["logits"] - st["logits"].amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        grad = -p * (g * p.gather(1, ids)).sum(1, keepdim=True)
        grad = grad.scatter_add(1, ids, g * p.gather(1, ids))
    else:
        if c["scoring"] == "softmax":
            e = torch.exp(l - l.amax(1, keepdim=True)) * has
            w = e / e.sum(1, keepdim=True).clamp(min=1e-30)
            d = w * (g - (g * w).sum(1, keepdim=True))
        else:
            e = torch.exp(-l.abs())
            s = torch.where(l >= 0, 1 / (1 + e), e / (1 + e)) * has
            slope = e / (1 + e) ** 2 * has
            if c["renorm"]:
                total = s.sum(1, keepdim=True) + 1e-20
                d = slope / total * (g - (g * s / total).sum(1, keepdim=True))
            else:
                d = slope * g
        grad = torch.zeros(M, E, device="cuda").scatter_add(1, ids, d)
    return {"dlogits": grad if st["base"] is None else grad + st["base"]}


def _e4m3(t):
    """fp64 values rounded to e4m3 (nearest, ties to even), as fp64."""
    t = t.clamp(-E4M3_MAX, E4M3_MAX)
    exponent = torch.frexp(t).exponent.clamp(min=-5) - 4  # of the last bit kept
    step = torch.exp2(exponent.double())
    return torch.round(t / step) * step


def _plain_norm(st):
    c = st["case"]
    M, N, q = c["M"], c["N"], c["quant"]
    h = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(st["res"].dtype)
    out = {} if st["res"] is None else {"h": h}
    f = h.double() if q else h.float()  # rounding to 8 bits tells apart values that lie close together
    r = 1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)
    y = f * r * st["w"].to(f.dtype)
    if c["keep"]:
        out["rstd"] = r[:, 0].float()
    if c["out"]:
        out["y"] = y.to(torch.bfloat16)
    if q:
        s = (y.view(M, N // q, q).abs().amax(2) / E4M3_MAX).float().clamp(min=TINY)
        out["q"] = _e4m3(y.view(M, N // q, q) / s.double()[:, :, None]).view(M, N).float().to(torch.float8_e4m3fn)
        out["scales"] = s
    return out


def _plain_norm_bwd(st):
    h, g, r = st["h"].float(), st["dy"].float(), st["r"][:, None]
    n = h * r
    wg = st["w"].float() * g
    dh = r * (wg - n * (wg * n).mean(1, keepdim=True))
    if st["dres"] is not None:
        dh = dh + st["dres"].float()
    return {"dh": dh.to(st["h"].dtype), "dw": (g * n).sum(0)}


def _plain_clip(st):
    total = torch.stack([t.double().square().sum() for t in st["grads"]]).sum()  # long sums: fp64
    norm = torch.sqrt(total)
    factor = torch.where(norm > st["max_norm"], st["max_norm"] / norm, 1.0).float()
    return {"norm": norm.float().view(1), "grads": [(t.float() * factor).to(t.dtype) for t in st["grads"]]}


# ------------------------------------------------------------------ the package's calls
def _moe():
    import int4_weight_only_moe_amd as moe
    return moe


def _own(st):
    moe, c = _moe(), st["case"]
    kept = st.setdefault("kept", {})  # output buffers and workspace, reused from call to call as a step loop does
    if c["op"] == "route":
        if not kept:
            kept["rb"] = moe.alloc_route_buffers(c["M"], c["E"], c["k"], c["block"] or 16)
        rb = moe.route_scored(st["logits"], kept["rb"], scoring=c["scoring"], bias=st["bias"], n_groups=c["G"],
                              top_groups=c["top_groups"], group_top=c["group_top"], renormalise=c["renorm"],
                              scale=c["scale"], row_valid=st["valid"], grouping=c["block"] > 0)
        out = {"ids": rb.topk_ids, "weights": rb.topk_weights}
        if c["block"]:
            out.update(rows=rb.sorted_token_ids, blocks=rb.block_expert_ids, offsets=rb.expert_offsets,
                       npp=rb.num_tokens_post_pad)
        return out
    if c["op"] == "route_bwd":
        kept["grad"] = moe.route_scored_backward(st["logits"], st["ids"], st["dweights"], scoring=c["scoring"],
                                                 renormalise=c["renorm"], scale=c["scale"], grad_base=st["base"],
                                                 grad_logits=kept.get("grad"))
        return {"dlogits": kept["grad"]}
    if c["op"] == "norm":
        if not kept:
            kept["bufs"] = moe.alloc_norm_buffers(c["M"], c["N"], None if st["res"] is None else st["res"].dtype,
                                                  out=c["out"], rstd=c["keep"], quant_group=c["quant"])
        bufs = moe.add_rms_norm(st["x"], st["w"], kept["bufs"], residual=st["res"], eps=EPS)
        out = {} if st["res"] is None else {"h": bufs.residual_out}
        if c["keep"]:
            out["rstd"] = bufs.rstd
        if c["out"]:
            out["y"] = bufs.out
        if c["quant"]:
            out.update(q=bufs.out8, scales=bufs.scales)
        return out
    if c["op"] == "norm_bwd":
        if not kept:
            kept["ws"] = torch.empty(moe.moe_add_rms_norm_workspace_bytes(c["M"], c["N"]), dtype=torch.uint8,
                                     device="cuda")
        kept["grads"] = moe.add_rms_norm_backward(st["dy"], st["h"], st["r"], st["w"], grad_residual=st["dres"],
                                                  grads=kept.get("grads"), workspace=kept["ws"])
        dh, dw = kept["grads"]
        return {"dh": dh, "dw": dw}
    if not kept:
        kept["out"] = [torch.empty_like(t) for t in st["grads"]]
        kept["ws"] = torch.empty(moe.moe_grad_norm_workspace_bytes(len(st["grads"])), dtype=torch.uint8, device="cuda")
    norm = moe.clip_grad_norm(st["grads"], st["max_norm"], out=kept["out"], workspace=kept["ws"])
    return {"norm": norm, "grads": kept["out"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "route_bwd": _plain_route_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd,
            "clip": _plain_clip}[state["case"]["op"]](state)


# ------------------------------------------------------------------ fp64
def _exact_weights(st):
    """The weights of each row's choice, with numpy: groups and experts are ranked by sorting their negatives."""
    c = st["case"]
    M, E, k, G = c["M"], c["E"], c["k"], c["G"]
    live = np.ones(M, bool) if st["valid"] is None else st["valid"].cpu().numpy()
    l = np.where(live[:, None], st["logits"].double().cpu().numpy(), 0.0)
    if c["scoring"] == "sigmoid":
        s = np.exp(-np.logaddexp(0.0, -l))
    else:
        s = np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))
    key = -(s + st["bias"].double().cpu().numpy()) if st["bias"] is not None else -s
    parts = key.reshape(M, G, E // G)
    sums = np.sort(parts, axis=2)[:, :, :c["group_top"]].sum(axis=2)
    rank = np.argsort(np.argsort(sums, axis=1, kind="stable"), axis=1, kind="stable")
    key = np.where((rank < c["top_groups"])[:, :, None], parts, np.inf).reshape(M, E)
    first = np.argsort(key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, first, axis=1)
    if c["renorm"]:
        w = w / w.sum(axis=1, keepdims=True)
    return torch.from_numpy(w * c["scale"] * live[:, None])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        out = {"ids": None, "weights": _exact_weights(st)}
        return {**out, "rows": None, "blocks": None, "offsets": None, "npp": None} if case["block"] else out
    if op == "route_bwd":
        has = st["ids"] >= 0
        l = st["logits"].double()
        member = torch.zeros(l.shape, dtype=torch.bool, device="cuda")
        dw = torch.zeros_like(l)
        for j in range(case["k"]):  # the rows' j-th choices
            rows = has[:, j].nonzero()[:, 0]
            at = st["ids"][rows, j].long()
            member[rows, at] = True
            dw[rows, at] = case["scale"] * st["dweights"][rows, j].double()
        if case["scoring"] == "softmax":
            kept = member if case["renorm"] else torch.ones_like(member)
            p = torch.softmax(torch.where(kept, l, -math.inf), 1).nan_to_num(0.0)
            grad = p * (dw - (dw * p).sum(1, keepdim=True))
        else:
            s = torch.sigmoid(l)
            if case["renorm"]:
                total = (s * member).sum(1, keepdim=True) + 1e-20
                dw = (dw - (dw * s).sum(1, keepdim=True) / total) / total
            grad = dw * s * torch.sigmoid(-l) * member
        return {"dlogits": grad if st["base"] is None else grad + st["base"].double()}
    if op == "norm":
        M, N, q = case["M"], case["N"], case["quant"]
        h = st["x"].double() if st["res"] is None else (st["x"].double() + st["res"].double()).to(st["res"].dtype).double()
        r = torch.rsqrt(h.pow(2).sum(1) / N + EPS)
        y = torch.einsum("mn,m,n->mn", h, r, st["w"].double())
        out = {} if st["res"] is None else {"h": h}
        if case["keep"]:
            out["rstd"] = r
        if case["out"]:
            out["y"] = y
        if q:
            s = torch.linalg.vector_norm(y.reshape(-1, q), ord=math.inf, dim=1) / E4M3_MAX
            s = s.to(torch.float32).double().clamp(min=TINY)
            out["q"] = (y.reshape(-1, q) / s[:, None]).reshape(M, N)
            out["scales"] = s.view(M, N // q)
        return out
    if op == "norm_bwd":
        N = case["N"]
        h, g, w = st["h"].double(), st["dy"].double(), st["w"].double()
        r = st["r"].double()
        along = torch.einsum("mn,mn,n->m", h, g, w)
        dh = (g * w) * r[:, None] - h * (r ** 3 * along / N)[:, None]
        if st["dres"] is not None:
            dh = dh + st["dres"].double()
        return {"dh": dh, "dw": torch.einsum("mn,mn,m->n", g, h, r)}
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t.double()) ** 2) for t in st["grads"]))
    factor = min(1.0, st["max_norm"] / norm)
    return {"norm": torch.tensor([norm], dtype=torch.float64), "grads": [t.double() * factor for t in st["grads"]]}
