"""Cases and plain forms of the operators beside the MoE layer's routing and
products: the balance loss of the router (per-expert counts, the loss and its
gradient) and low-rank adapters of many requests beside a shared projection
(forward and backward).

`run` computes a case with elementary torch operations in fp32, or, with
`own` set, with the calls a user makes of the package. `exact` computes the
same outputs in fp64 from the definitions.

Balance loss, for each sequence s of T valid tokens (p = softmax of a token's
logits over the E experts, c = how often each expert was chosen; c and the
sums of p are returned too):
    loss_s = E / (k T^2) * sum_e c[s, e] * sum_t p[t, e]
    dloss_s / dlogits[t, e] = E / (k T^2) * p[t, e] * (c[s, e] - sum_j c[s, j] p[t, j])
Adapters, for a token t of a request with adapter a (A [r, K], B [N, r], scale s):
    h_t = A_a x_t        out_t = base_t + s_a B_a h_t
    dh_t = s_a B_a^T dout_t        dx_t = dxbase_t + A_a^T dh_t
    dA_a = sum_t dh_t x_t^T        dB_a = s_a sum_t dout_t h_t^T
A token without an adapter has out_t = base_t and dx_t = dxbase_t.
"""
import math
import random

import torch

own = False

HIDDEN, INTER, EXPERTS = 7168, 2048, 384  # the 384-expert layer of the package's workloads


def _balance(name, back, M, E, k, S, masked):
    return {"name": name, "op": "balance", "back": back, "M": M, "E": E, "k": k, "S": S, "masked": masked}


def _lora(name, back, M, K, N, r, L, R, fp32=False, save=False, mixed=False):
    return {"name": name, "op": "lora", "back": back, "M": M, "K": K, "N": N, "r": r, "L": L, "R": R, "fp32": fp32,
            "save": save, "mixed": mixed}


def listed():
    return [
        # a small layer's step of a few tokens: latency
        _balance("balance_fwd_few", False, 48, 8, 2, 1, False),
        # a training batch of four packed sequences with padding, 384 experts
        _balance("balance_fwd_batch", False, 16384, EXPERTS, 8, 4, True),
        # the most experts the routing takes, one long batch
        _balance("balance_fwd_wide", False, 32768, 1024, 8, 1, False),
        # the backward pass of the packed batch
        _balance("balance_bwd_batch", True, 16384, EXPERTS, 8, 4, True),
        # odd sizes: an expert count that is no multiple of the wave
        _balance("balance_bwd_odd", True, 4099, 60, 4, 3, False),
        # one stream decoding with its adapter
        _lora("lora_fwd_one_token", False, 1, HIDDEN, HIDDEN, 16, 8, 1),
        # 64 streams decoding, nearly each with an adapter of its own
        _lora("lora_fwd_decode", False, 64, HIDDEN, HIDDEN, 16, 96, 64, mixed=True),
        # prompts of six requests in one batch
        _lora("lora_fwd_prompts", False, 4096, HIDDEN, HIDDEN, 64, 32, 6),
        # adapters of the router's projection (fp32 logits) in training: h is kept for the backward pass
        _lora("lora_fwd_router", False, 2051, HIDDEN, EXPERTS, 8, 32, 40, fp32=True, save=True),
        # one adapter trained on a long batch
        _lora("lora_bwd_one", True, 8192, HIDDEN, HIDDEN, 64, 1, 1),
        # eight adapters trained at once, an odd batch, a narrower projection
        _lora("lora_bwd_many", True, 1999, HIDDEN, INTER, 16, 8, 12),
        # the router's adapters, fp32 gradients of the logits
        _lora("lora_bwd_router", True, 1023, HIDDEN, EXPERTS, 32, 4, 5, fp32=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    if rng.random() < 0.4:
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, EXPERTS, 512, rng.randint(9, 1024), 1024])
        M = _log(rng, 1, min(32768, 32768 * 1024 // E))
        return {"op": "balance", "back": rng.random() < 0.5, "M": M, "E": E, "k": rng.randint(1, min(8, E)),
                "S": _log(rng, 1, min(16, M)), "masked": rng.random() < 0.5}
    back = rng.random() < 0.5
    fp32 = rng.random() < 0.3
    K = rng.choice([512, 1024, INTER, 4096, HIDDEN, 8 * rng.randint(16, 896)])
    N = rng.choice([8, 60, 64, 129, 256, EXPERTS, 1000]) if fp32 else rng.choice(
        [512, 1024, INTER, 4096, HIDDEN, 8 * rng.randint(16, 896)])
    M = _log(rng, 1, 8192 if back else 4096)
    R = _log(rng, 1, min(M, 256))
    # the largest ranks go with fewer tokens, so that no case costs more than the listed ones
    r = rng.choice([8, 16, 24, 32, 64] if M > 2048 else [8, 16, 32, 48, 64, 128])
    L = _log(rng, 1, 64 if r <= 32 else 16)
    return {"op": "lora", "back": back, "M": M, "K": K, "N": N, "r": r, "L": L, "R": R, "fp32": fp32,
            "save": not back and rng.random() < 0.5, "mixed": rng.random() < 0.5}


def _requests(case):
    """(requests with an adapter, distinct adapters): every eighth request has none."""
    n = case["R"] - case["R"] // 8
    return n, min(n, case["L"])


def work(case):
    M = case["M"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        small = (M if case["masked"] else 0) + 4 * (S + 1)
        if case["back"]:
            return {"bytes": 8.0 * M * E + 4.0 * S * E + 8 * S + small, "flops": 7.0 * M * E}
        return {"bytes": 4.0 * M * E + 4.0 * M * k + 8.0 * S * E + 8 * S + small, "flops": 5.0 * M * E}
    K, N, r, L = case["K"], case["N"], case["r"], case["L"]
    y = 4 if case["fp32"] else 2
    _, D = _requests(case)
    weights = 2.0 * D * r * (K + N) + 4 * L
    if not case["back"]:
        h = 4.0 * M * r if case["save"] else 0.0
        return {"bytes": 2.0 * M * K + 2.0 * y * M * N + weights + h + 4 * M, "flops": 2.0 * M * r * (K + N)}
    grads = 4.0 * L * r * (K + N)
    return {"bytes": y * M * N + 6.0 * M * K + 4.0 * M * r + weights + grads + 4 * M,
            "flops": 4.0 * M * r * (K + N)}


def _cuts(g, M, R):
    """R + 1 ascending offsets of ragged, non-empty pieces of M rows (a host tensor)."""
    inner = torch.randperm(M - 1, generator=g)[: R - 1].sort().values + 1 if R > 1 else torch.empty(0, dtype=torch.int64)
    return torch.cat([torch.zeros(1, dtype=torch.int64), inner, torch.tensor([M])])


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    M = case["M"]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(dtype)

    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        logits = normal(M, E) + 0.7 * normal(1, E)  # some experts are liked more than others
        st = {"case": case, "logits": logits, "topk_ids": logits.topk(k, dim=1).indices.to(torch.int32).contiguous(),
              "offsets": _cuts(host, M, S).to(torch.int32).cuda(), "valid": None}
        if case["masked"]:  # padding rows hold whatever was left there
            st["valid"] = torch.rand(M, generator=g, device="cuda") > 0.1
            logits[~st["valid"]] = float("nan")
        if case["back"]:
            counts, tokens = _balance_counts(st)
            st["counts"], st["tokens"] = counts, tokens
            st["dloss"] = normal(S, scale=0.01)
        return st
    K, N, r, L, R = (case[n] for n in ("K", "N", "r", "L", "R"))
    dt = torch.float32 if case["fp32"] else torch.bfloat16
    with_adapter, _ = _requests(case)
    order = torch.randperm(L, generator=host)
    of_request, n = [], 0
    for i in range(R):
        if i % 8 == 7:
            of_request.append(-1)
        else:
            of_request.append(int(order[n % L]))
            n += 1
    cuts = _cuts(host, M, R)
    ids = torch.tensor(of_request).repeat_interleave(cuts[1:] - cuts[:-1])
    if case["mixed"]:
        ids = ids[torch.randperm(M, generator=host)]
    st = {"case": case, "x": normal(M, K, dtype=torch.bfloat16), "ids": ids.to(torch.int32).cuda(),
          "a": normal(L, r, K, scale=K ** -0.5, dtype=torch.bfloat16),
          "b": normal(L, N, r, scale=0.5 * r ** -0.5, dtype=torch.bfloat16),
          "scales": 0.5 + torch.rand(L, generator=g, device="cuda")}
    if case["back"]:
        st["dout"] = normal(M, N, scale=0.02, dtype=dt)
        st["dx_base"] = normal(M, K, scale=0.02, dtype=torch.bfloat16)
        st["h"] = _down(st)
    else:
        st["base"] = normal(M, N, dtype=dt)
    return st


# ------------------------------------------------------------------ plain forms
def _rows(st):
    """(row numbers, the row's sequence) of a balance case."""
    rows = torch.arange(st["logits"].shape[0], device="cuda")
    return rows, torch.bucketize(rows, st["offsets"][1:].long(), right=True)


def _balance_counts(st):
    S, E = st["case"]["S"], st["case"]["E"]
    M, k = st["topk_ids"].shape
    rows, seq = _rows(st)
    live = torch.ones(M, dtype=torch.bool, device="cuda") if st["valid"] is None else st["valid"]
    flat = (seq[:, None] * E + st["topk_ids"].long()).reshape(-1)
    counts = torch.zeros(S * E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, flat, live[:, None].expand(M, k).reshape(-1).to(torch.int32))
    tokens = torch.zeros(S, dtype=torch.int32, device="cuda").scatter_add_(0, seq, live.to(torch.int32))
    return counts.view(S, E), tokens


def _probs(st):
    logits = st["logits"]
    if st["valid"] is not None:
        logits = torch.where(st["valid"][:, None], logits, torch.zeros((), device="cuda"))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    return p if st["valid"] is None else p * st["valid"][:, None]


def _plain_balance(st):
    E, k, S = (st["case"][n] for n in ("E", "k", "S"))
    if st["case"]["back"]:
        _, seq = _rows(st)
        p, c = _probs(st), st["counts"].float()[seq]
        t = st["tokens"].float().clamp(min=1)
        w = (st["dloss"] * E / (k * t * t))[seq][:, None]
        return {"dlogits": w * p * (c - (c * p).sum(1, keepdim=True))}
    counts, tokens = _balance_counts(st)
    _, seq = _rows(st)
    member = (seq[None, :] == torch.arange(S, device="cuda")[:, None]).float()
    t = tokens.float().clamp(min=1)
    sums = member @ _probs(st)
    loss = (counts.float() * sums).sum(1) * E / (k * t * t)
    return {"loss": loss, "counts": counts, "prob_sums": sums, "tokens": tokens}


def _picked(st):
    """(row numbers, adapter or 0, 1.0 where the row has one)."""
    ids = st["ids"].long()
    L = st["case"]["L"]
    return torch.arange(ids.numel(), device="cuda"), ids.clamp(0, L - 1), ((ids >= 0) & (ids < L)).float()


def _by_row(st):
    """Whether the plain form gathers each row's adapter (few rows) or multiplies by all adapters and picks."""
    c = st["case"]
    return c["M"] * c["r"] * max(c["K"], c["N"]) <= 1 << 27


def _down(st):
    rows, a, has = _picked(st)
    L, r, K = st["a"].shape
    x = st["x"].float()
    if _by_row(st):
        h = torch.bmm(st["a"][a].float(), x[:, :, None])[:, :, 0]
    else:
        h = (x @ st["a"].float().view(L * r, K).t()).view(-1, L, r)[rows, a]
    return h * has[:, None]


def _spread(st, v):
    """[M, r] values to [M, L * r], each row's at its adapter's place."""
    rows, a, has = _picked(st)
    full = torch.zeros(v.shape[0], st["case"]["L"], v.shape[1], device="cuda")
    full[rows, a] = v * has[:, None]
    return full.view(v.shape[0], -1)


def _plain_lora(st):
    rows, a, has = _picked(st)
    L, r, K = st["a"].shape
    N = st["b"].shape[1]
    s = (st["scales"][a] * has)[:, None]
    if not st["case"]["back"]:
        h = _down(st)
        if _by_row(st):
            d = torch.bmm(st["b"][a].float(), (h * s)[:, :, None])[:, :, 0]
        else:
            d = _spread(st, h * s) @ st["b"].float().permute(0, 2, 1).reshape(L * r, N)
        out = {"out": (st["base"].float() + d).to(st["base"].dtype)}
        return {**out, "h": h} if st["case"]["save"] else out
    g = st["dout"].float()
    if _by_row(st):
        dh = torch.bmm(g[:, None, :], st["b"][a].float())[:, 0] * s
        dx = torch.bmm(dh[:, None, :], st["a"][a].float())[:, 0]
        wide = _spread(st, dh)
    else:
        dh = (g @ st["b"].float().permute(0, 2, 1).reshape(L * r, N).t()).view(-1, L, r)[rows, a] * s
        wide = _spread(st, dh)
        dx = wide @ st["a"].float().view(L * r, K)
    da = (wide.t() @ st["x"].float()).view(L, r, K)
    db = (_spread(st, st["h"] * s).t() @ g).view(L, r, N).permute(0, 2, 1).contiguous()
    return {"dx": (st["dx_base"].float() + dx).to(torch.bfloat16), "da": da, "db": db}


# ------------------------------------------------------------------ the package's calls
def _moe():
    import int4_weight_only_moe_amd as moe
    return moe


def _own(st):
    moe, c = _moe(), st["case"]
    kept = st.setdefault("kept", {})  # output buffers and workspace, reused from call to call as a step loop does
    if c["op"] == "balance":
        if c["back"]:
            kept["grad"] = moe.balance_loss_backward(st["logits"], c["k"], st["counts"], st["tokens"], st["dloss"],
                                                     seq_offsets=st["offsets"], row_valid=st["valid"],
                                                     grad_logits=kept.get("grad"))
            return {"dlogits": kept["grad"]}
        if not kept:
            kept["bufs"] = moe.alloc_balance_buffers(c["M"], c["E"], c["S"])
        bufs = moe.balance_loss(st["logits"], st["topk_ids"], kept["bufs"], seq_offsets=st["offsets"],
                                row_valid=st["valid"])
        return {"loss": bufs.loss, "counts": bufs.expert_counts, "prob_sums": bufs.prob_sums, "tokens": bufs.seq_tokens}
    if not kept:
        kept["ws"] = torch.empty(moe.moe_lora_workspace_bytes(c["M"], c["L"], c["K"], c["N"], c["r"], c["back"]),
                                 dtype=torch.uint8, device="cuda")
    if c["back"]:
        kept["grads"] = moe.lora_backward(st["dout"], st["x"], st["ids"], st["h"], st["a"], st["b"], st["scales"],
                                          dx_base=st["dx_base"], grads=kept.get("grads"), workspace=kept["ws"])
        dx, da, db = kept["grads"]
        return {"dx": dx, "da": da, "db": db}
    if c["save"] and "h" not in kept:
        kept["h"] = torch.empty(c["M"], c["r"], device="cuda")
    kept["out"] = moe.lora_forward(st["x"], st["ids"], st["a"], st["b"], st["scales"], base=st["base"],
                                   out=kept.get("out"), h=kept.get("h"), workspace=kept["ws"])
    return {"out": kept["out"], "h": kept["h"]} if c["save"] else {"out": kept["out"]}


def run(state):
    if own:
        return _own(state)
    return _plain_balance(state) if state["case"]["op"] == "balance" else _plain_lora(state)


# ------------------------------------------------------------------ fp64
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        logits = st["logits"].double()
        cuts = st["offsets"].tolist()
        losses, sums, grad = [], [], torch.zeros_like(logits)
        for s in range(S):
            rows = torch.arange(cuts[s], cuts[s + 1], device="cuda")
            if st["valid"] is not None:
                rows = rows[st["valid"][rows]]
            T = max(1, rows.numel())
            p = torch.softmax(logits[rows], 1)
            f = torch.bincount(st["topk_ids"][rows].long().reshape(-1), minlength=E).double() / (k * T)
            losses.append(E * (f * p.sum(0) / T).sum())
            sums.append(p.sum(0))
            if case["back"]:
                dp = (E / T) * f * st["dloss"][s].double()  # d loss / d p, the same for each row
                grad[rows] = p * (dp - (p * dp).sum(1, keepdim=True))
        if case["back"]:
            return {"dlogits": grad}
        return {"loss": torch.stack(losses), "counts": None, "prob_sums": torch.stack(sums), "tokens": None}
    x, ids = st["x"].double(), st["ids"]
    if case["back"]:
        dout, h = st["dout"].double(), st["h"].double()
        dx = st["dx_base"].double()
        da, db = torch.zeros(st["a"].shape, dtype=torch.float64, device="cuda"), torch.zeros(
            st["b"].shape, dtype=torch.float64, device="cuda")
        for i in range(case["L"]):
            rows = (ids == i).nonzero()[:, 0]
            A, B, s = st["a"][i].double(), st["b"][i].double(), st["scales"][i].double()
            dh = s * (dout[rows] @ B)
            dx[rows] += dh @ A
            da[i] = dh.t() @ x[rows]
            db[i] = s * (dout[rows].t() @ h[rows])
        return {"dx": dx, "da": da, "db": db}
    out = st["base"].double()
    hs = torch.zeros(case["M"], case["r"], dtype=torch.float64, device="cuda")
    for i in range(case["L"]):
        rows = (ids == i).nonzero()[:, 0]
        h = x[rows] @ st["a"][i].double().t()
        hs[rows] = h
        out[rows] += st["scales"][i].double() * (h @ st["b"][i].double().t())
    return {"out": out, "h": hs} if case["save"] else {"out": out}
