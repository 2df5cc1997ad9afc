"""Measured cases of the operators around the expert layer's backward pass.

A pre-norm expert block's training step runs, next to ``moe_bwd``: the layer norm in front of the block
and its backward pass, the router's top-K with the load-balance and z losses and their gradient, and the
gated activation that saves the gate/up checkpoint in 8 bits, which ``moe_bwd`` then reads.  Each case is
one call (or the pair of calls) that a training program makes:

  ln_fwd / ln_bwd    layer_norm_fwd / layer_norm_bwd
  router / balance   router_fwd with the balance losses / balance_bwd
  pack               glu_fwd writing the 8-bit checkpoint, ckpt8_unpack reading it back
  moe_bwd8           moe_bwd on an 8-bit checkpoint

``run`` computes the plain form in elementary torch operations, or, where ``own`` is true, calls the
library.  ``exact`` gives the same outputs in 64 bits, the gradients by automatic differentiation.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
ALPHA, BETA = 0.01, 0.001
NEG_INF = float("-inf")
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a norm on the few rows of an interactive step: launch latency
        {"name": "ln_fwd_few_rows", "op": "ln_fwd", "T": 7, "H": 2048, "type": "bf16", "kind": "layer", "skip": True},
        # the norm before the imbalanced workload's block, the residual stream updated in the same pass
        {"name": "ln_fwd_large", "op": "ln_fwd", "T": 65536, "H": 4096, "type": "bf16", "kind": "layer", "skip": True},
        # an fp32 residual stream of odd width: rows that are not 16-byte aligned
        {"name": "ln_bwd_odd_fp32", "op": "ln_bwd", "T": 4099, "H": 1111, "type": "fp32", "kind": "layer", "skip": False},
        # that norm's backward on the imbalanced workload, the skip connection's gradient added
        {"name": "ln_bwd_large", "op": "ln_bwd", "T": 65536, "H": 4096, "type": "bf16", "kind": "layer", "skip": True},
        # routing of a small batch: one short sequence of the fine-grained workload's router
        {"name": "router_small", "op": "router", "T": 37, "E": 64, "K": 8, "S": 1, "mode": 0, "renorm": False},
        # the imbalanced workload's router on a packed batch of sequences of different lengths
        {"name": "router_large", "op": "router", "T": 65536, "E": 128, "K": 8, "S": 48, "mode": 1, "renorm": True},
        # loss gradient on the fine-grained workload's router, one global balance loss
        {"name": "balance_global", "op": "balance", "T": 16384, "E": 64, "K": 8, "S": 1, "add": False},
        # loss gradient per packed sequence, added to the router's own gradient, many experts
        {"name": "balance_packed", "op": "balance", "T": 131072, "E": 256, "K": 8, "S": 61, "add": True},
        # the tiny workload's activation and checkpoint
        {"name": "pack_tiny", "op": "pack", "T": 256, "I": 256, "E": 4, "K": 2, "B": 128},
        # the fine-grained workload's activation and checkpoint: 131,072 routed rows
        {"name": "pack_large", "op": "pack", "T": 16384, "I": 1024, "E": 64, "K": 8, "B": 128},
        # the tiny workload's backward from an 8-bit checkpoint
        {"name": "moe_bwd8_tiny", "op": "moe_bwd8", "T": 256, "H": 128, "I": 256, "E": 4, "K": 2, "B": 128},
        # a training micro-batch's backward from an 8-bit checkpoint
        {"name": "moe_bwd8_train", "op": "moe_bwd8", "T": 4096, "H": 1024, "I": 512, "E": 32, "K": 8, "B": 128},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "router", "balance", "pack", "moe_bwd8"])
    if op in ("ln_fwd", "ln_bwd"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            H = -(-H // 64) * 64
        kind = rng.choice(["layer", "rms"])
        kind_type = rng.choice(["bf16", "fp32"])
        most = 65536 * 4096 // (2 if kind_type == "fp32" else 1) // H
        return {"op": op, "T": _log_int(rng, 1, min(131072, most)), "H": H, "type": kind_type, "kind": kind,
                "skip": rng.random() < 0.5}
    if op in ("router", "balance"):
        E = rng.choice([_log_int(rng, 4, 512), 8 * rng.randint(1, 32)])
        K = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 131072 * 256 // max(E, 256))
        case = {"op": op, "T": T, "E": E, "K": K, "S": rng.randint(1, max(1, min(64, T // 4)))}
        return dict(case, mode=rng.randint(0, 2), renorm=rng.random() < 0.5) if op == "router" else dict(case, add=rng.random() < 0.5)
    E = rng.randint(2, 48)
    K = rng.randint(1, min(8, E))
    B = rng.choice([128, 256, 512])
    if op == "pack":
        I = 128 * rng.randint(1, 12)
        T = _log_int(rng, 16, min(16384, 16384 * 8 * 1024 // (K * I)))
        return {"op": op, "T": T, "I": I, "E": E, "K": K, "B": B}
    H, I = 128 * rng.randint(1, 8), 128 * rng.randint(1, 4)
    return {"op": op, "T": _log_int(rng, 16, 4096), "H": H, "I": I, "E": min(E, 32), "K": K, "B": B}


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _segments(T, S, seed):
    """Offsets of S packed sequences in T token slots: different lengths, an empty sequence where there are
    several, and a few padding tokens behind the last."""
    gen = torch.Generator().manual_seed(seed + 1)
    end = T - T // 50
    cuts = torch.sort(torch.randint(0, end + 1, (max(S - 1, 0),), generator=gen)).values
    if S >= 3:
        cuts[1] = cuts[0]
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([end])]).to(DEV, torch.int32)


def _logits(T, E, gen):
    """Router logits of uneven experts; some experts masked for some tokens, one token with none left."""
    logits = torch.randn(T, E, generator=gen, device=DEV)
    logits += torch.randn(E, generator=gen, device=DEV)
    logits[:: 97, E // 2] = NEG_INF
    if T > 5:
        logits[5] = NEG_INF
    return logits


def _blocks(T, K, E, B):
    """Blocks of the checkpoint layout that any routing of T * K rows needs at most."""
    left = T * K - (E - 1)
    return T * K if left <= 0 else -(-left // B) + E - 1


def _routing(T, K, E, B, gen):
    """Top-K routing of T tokens, and where its rows lie: grouped by expert, and in blocks of B slots."""
    p = torch.softmax(torch.randn(T, E, generator=gen, device=DEV), dim=-1)
    s, ids = torch.topk(p, K, dim=-1)
    s = (s / s.sum(-1, keepdim=True)).contiguous()
    ids = ids.to(torch.int32).contiguous()
    flat = ids.flatten().long()
    count = torch.bincount(flat, minlength=E)
    first = torch.cumsum(count, 0) - count
    per = (count + B - 1) // B
    first_block = torch.cumsum(per, 0) - per
    order = torch.argsort(flat, stable=True)
    expert = flat[order]
    place = torch.arange(T * K, device=DEV) - first[expert]
    N = _blocks(T, K, E, B)
    block_to_expert = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    block_to_expert[: int(per.sum())] = torch.repeat_interleave(torch.arange(E, device=DEV), per).int()
    end = lambda first, total: torch.cat([first, total.reshape(1)]).to(torch.int32)  # noqa: E731
    meta = {"expert_offsets": end(first, count.sum()), "block_offsets": end(first_block, per.sum()),
            "block_to_expert": block_to_expert, "s_scatter_idx": order.to(torch.int32)}
    return {"s": s, "ids": ids, "route_meta": meta, "order": order, "expert": expert, "place": place,
            "slot": first_block[expert] * B + place, "capacity": int(count.max()), "N": N}


def _pack(h):
    """8-bit codes and scale bytes of pre-activations h [N, 2, I, B]: groups of 32 slots of one feature share
    the power of two 2^(byte - 127), the codes are integers of at most 127.  The bytes are laid out
    [N, 2, B/128, I/32, 4, 32]: 128 slots, 32 features, group, feature."""
    N, two, I, B = h.shape
    g = h.float().reshape(N, two, I, B // 32, 32)
    exponent = torch.frexp(g.abs().amax(-1))[1] - 1 + 127          # exponent field of the largest magnitude
    byte = (exponent - 6).clamp(1, 254)
    q = torch.round(torch.ldexp(g, (127 - byte)[..., None])).clamp(-127, 127)
    scales = byte.reshape(N, two, I // 32, 32, B // 128, 4).permute(0, 1, 4, 2, 5, 3)
    return q.reshape(N, two, I, B).to(torch.int8), scales.contiguous().to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if op in ("ln_fwd", "ln_bwd"):
        T, H, dt = case["T"], case["H"], TYPES[case["type"]]
        x = (rand(T, H) + 0.5 * rand(H)).to(dt)
        st = {"x": x, "gamma": 1 + 0.1 * rand(H), "beta": 0.1 * rand(H)}
        if op == "ln_fwd":
            st["residual"] = rand(T, H).to(dt) if case["skip"] else None
        else:
            st["dy"] = rand(T, H).to(dt)
            st["dres"] = rand(T, H).to(dt) if case["skip"] else None
            xf = x.float()
            mean = xf.mean(-1) if case["kind"] == "layer" else torch.zeros(T, device=DEV)
            st["mean"], st["rstd"] = mean, torch.rsqrt((xf - mean[:, None]).square().mean(-1) + EPS)
    elif op in ("router", "balance"):
        T, E, K = case["T"], case["E"], case["K"]
        st = {"logits": _logits(T, E, gen), "seg": _segments(T, case["S"], seed)}
        if op == "balance":
            fwd = _plain_router(st, dict(case, mode=2, renorm=False))
            st.update(lse=fwd["lse"], counts=fwd["counts"], dloss=1 + 0.5 * rand(2))
            st["add"] = rand(T, E) * 1e-3 if case["add"] else None
    else:
        T, I, E, K, B = (case[k] for k in ("T", "I", "E", "K", "B"))
        st = _routing(T, K, E, B, gen)
        if op == "pack":
            st["h"] = (rand(T * K, 2 * I) * (0.5 + rand(2 * I).abs())).to(torch.bfloat16)
        else:
            H = case["H"]
            st["x"], st["dout"] = rand(T, H).to(torch.bfloat16), rand(T, H).to(torch.bfloat16)
            st["W1"] = (rand(E, H, 2 * I) * 0.02).to(torch.bfloat16)
            st["W2"] = (rand(E, I, H) * 0.02).to(torch.bfloat16)
            st["q"], st["sf"] = _pack((rand(st["N"], 2, I, B) * (0.02 * math.sqrt(H))).to(torch.bfloat16))
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------------------------------------------
# plain forms: 32-bit torch operations
# ---------------------------------------------------------------------------------------------------
def _plain_ln_fwd(st, c):
    dt = st["x"].dtype
    s = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(dt)
    sf = s.float()
    mean = sf.mean(-1) if c["kind"] == "layer" else torch.zeros(c["T"], device=DEV)
    d = sf - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + EPS)
    y = d * rstd[:, None] * st["gamma"]
    if c["kind"] == "layer":
        y = y + st["beta"]
    out = {"y": y.to(dt), "rstd": rstd}
    if c["kind"] == "layer":
        out["mean"] = mean
    if st["residual"] is not None:
        out["sum"] = s
    return out


def _plain_ln_bwd(st, c):
    x, dy = st["x"].float(), st["dy"].float()
    xh = (x - st["mean"][:, None]) * st["rstd"][:, None]
    w = dy * st["gamma"]
    d = w - xh * (w * xh).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        d = d - w.mean(-1, keepdim=True)
    d = d * st["rstd"][:, None]
    if st["dres"] is not None:
        d = d + st["dres"].float()
    out = {"dx": d.to(st["x"].dtype), "dgamma": (dy * xh).sum(0)}
    if c["kind"] == "layer":
        out["dbeta"] = dy.sum(0)
    return out


def _in_segment(st, c):
    """[S, T]: 1 where token t belongs to sequence s."""
    t = torch.arange(c["T"], device=DEV)
    return ((t >= st["seg"][:-1, None]) & (t < st["seg"][1:, None])).float()


def _plain_router(st, c):
    logits, T, E, K = st["logits"], c["T"], c["E"], c["K"]
    member = _in_segment(st, c)
    valid = member.sum(0) > 0
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :K], ids[:, :K]
    used = valid[:, None] & (top > NEG_INF)
    m = logits.amax(-1, keepdim=True)
    base = torch.where(m > NEG_INF, m, torch.zeros_like(m))
    e = torch.exp(logits - base)
    total = e.sum(-1, keepdim=True)
    lse = (base + torch.log(total))[:, 0]
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    if c["mode"] == 2:
        scores = top
    else:  # the softmax over the selected logits is the renormalised top-K of the softmax, too
        se = torch.exp(top - base)
        scores = se / (total if c["mode"] == 1 and not c["renorm"] else se.sum(-1, keepdim=True))
    scores = torch.where(used, scores, torch.zeros_like(scores))
    ids = torch.where(used, ids, torch.full_like(ids, -1)).to(torch.int32)
    picked = torch.zeros(T, E + 1, device=DEV).scatter_(1, torch.where(used, ids.long(), E), 1.0)[:, :E]
    counts = member @ picked
    prob = member @ p
    length = member.sum(1)
    n = length.sum().clamp(min=1)
    per = (counts * prob).sum(1) / length.clamp(min=1)
    lse = torch.where(valid, lse, torch.full_like(lse, NEG_INF))
    z = torch.where(lse > NEG_INF, lse, torch.zeros_like(lse))
    loss = torch.stack([ALPHA * E / (K * n) * per.sum(), BETA / n * (z * z).sum()])
    return {"scores": scores, "ids": ids, "lse": lse, "counts": counts.to(torch.int32), "prob_sum": prob, "loss": loss}


def _plain_balance(st, c):
    member = _in_segment(st, c)
    length = member.sum(1)
    n = length.sum().clamp(min=1)
    lse = st["lse"][:, None]
    live = lse > NEG_INF
    p = torch.where(live, torch.exp(st["logits"] - torch.where(live, lse, torch.zeros_like(lse))), 0.0)
    scale = member.T @ (1 / length.clamp(min=1))[:, None] * (ALPHA * c["E"] / (c["K"] * n)) * st["dloss"][0]
    cnt = member.T @ st["counts"].float()
    d = scale * p * (cnt - (cnt * p).sum(-1, keepdim=True))
    d = d + (st["dloss"][1] * 2 * BETA / n) * torch.where(live, lse, torch.zeros_like(lse)) * p
    return d if st["add"] is None else st["add"] + d


def _plain_pack(st, c):
    I, B = c["I"], c["B"]
    h = st["h"].float()
    g, u = h[:, :I], h[:, I:]
    a = g / (1 + torch.exp(-g)) * u
    slots = torch.zeros(st["N"] * B, 2 * I, device=DEV)
    slots[st["slot"]] = h
    groups = slots.reshape(-1, 32, 2 * I)
    exponent = torch.frexp(groups.abs().amax(1, keepdim=True))[1] - 1
    step = torch.clamp(exponent - 6, min=-126)
    q = torch.round(torch.ldexp(groups, -step)).clamp(-127, 127)
    values = torch.ldexp(q, step).reshape(-1, 2 * I)[st["slot"]]
    return {"a": a.to(torch.bfloat16), "h": values.to(torch.bfloat16)}


def _plain_moe_bwd8(st, c):
    T, H, I, E, K, B = (c[k] for k in ("T", "H", "I", "E", "K", "B"))
    cap = st["capacity"]
    scale = st["sf"].float().permute(0, 1, 3, 5, 2, 4).reshape(st["N"], 2, I, B // 32)
    h = st["q"].float().reshape(st["N"], 2, I, B // 32, 32) * torch.exp2(scale - 127)[..., None]
    h = h.reshape(st["N"], 2 * I, B).transpose(1, 2).reshape(-1, 2 * I)[st["slot"]]
    at = st["expert"] * cap + st["place"]                # each grouped row's place in [E, cap]
    token = st["order"] // K
    padded = lambda rows: torch.zeros(E * cap, rows.shape[1], device=DEV).index_copy_(0, at, rows).reshape(E, cap, -1)  # noqa: E731
    xg, dg = padded(st["x"].float()[token]), padded(st["dout"].float()[token])
    W1, W2 = st["W1"].float(), st["W2"].float()
    s = st["s"].flatten()[st["order"]][:, None]
    dA_raw = torch.bmm(dg, W2.transpose(1, 2)).reshape(E * cap, I)[at]
    gate, up = h[:, :I], h[:, I:]
    sig = 1 / (1 + torch.exp(-gate))
    a = gate * sig * up
    ds = torch.zeros(T * K, device=DEV).index_copy_(0, st["order"], (dA_raw * a).sum(-1)).reshape(T, K)
    dA = s * dA_raw
    dh = torch.cat([dA * up * sig * (1 + gate * (1 - sig)), dA * gate * sig], 1)
    dh_p = padded(dh)
    dW2 = torch.bmm(padded(s * a).transpose(1, 2), dg)
    dW1 = torch.bmm(xg.transpose(1, 2), dh_p)
    dx_rows = torch.bmm(dh_p, W1.transpose(1, 2)).reshape(E * cap, H)[at]
    back = torch.empty(T * K, H, device=DEV).index_copy_(0, st["order"], dx_rows)
    bf = torch.bfloat16
    return {"dx": back.reshape(T, K, H).sum(1).to(bf), "dW1": dW1.to(bf), "dW2": dW2.to(bf), "ds": ds}


PLAIN = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "router": _plain_router, "balance": _plain_balance,
         "pack": _plain_pack, "moe_bwd8": _plain_moe_bwd8}


# ---------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------
def _own(st, c):
    import moe_expert_layer_routing_gb300 as mb
    op = c["op"]
    if op in ("ln_fwd", "ln_bwd"):
        layer = c["kind"] == "layer"
        kind = mb.NORM_LAYER if layer else mb.NORM_RMS
        if op == "ln_fwd":
            r = mb.layer_norm_fwd(st["x"], st["gamma"], st["beta"] if layer else None, eps=EPS,
                                  residual=st["residual"], kind=kind)
            keys = ["y", "rstd"] + ["mean"] * layer + ["sum"] * (st["residual"] is not None)
        else:
            r = mb.layer_norm_bwd(st["dy"], st["x"], st["gamma"], st["mean"] if layer else None, st["rstd"],
                                  dres=st["dres"], kind=kind)
            keys = ["dx", "dgamma"] + ["dbeta"] * layer
        return {k: r[k] for k in keys}
    if op == "router":
        r = mb.router_fwd(c["mode"], st["logits"], c["K"], renorm=c["renorm"], seg_offsets=st["seg"], alpha=ALPHA, beta=BETA)
        return {k: r[k] for k in ("scores", "ids", "lse", "counts", "prob_sum", "loss")}
    if op == "balance":
        return mb.balance_bwd(st["logits"], st["lse"], st["counts"], c["K"], seg_offsets=st["seg"], alpha=ALPHA,
                              beta=BETA, dloss=st["dloss"], add=st["add"])
    if op == "pack":
        r = mb.glu_fwd(st["h"], st["route_meta"], c["B"])
        return {"a": r["a"], "h": mb.ckpt8_unpack(r["ckpt_q"], r["ckpt_sf"], st["route_meta"], st["h"].shape[0])}
    r = mb.moe_bwd(x=st["x"], dout=st["dout"], s=st["s"], ids=st["ids"], E=c["E"], I=c["I"], block_size=c["B"],
                   ckpt_q=st["q"], ckpt_sf=st["sf"], W1=st["W1"], W2=st["W2"])
    return {k: r[k] for k in ("dx", "dW1", "dW2", "ds")}


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------------------------------
def exact(case, seed):
    st, c = prepare(case, seed), case
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    op = c["op"]
    layer = c.get("kind") == "layer"

    def norm(x, gamma, beta, mean, rstd):
        y = (x - mean) * rstd * gamma
        return y + beta if layer else y

    def moments(x):
        mean = x.sum(-1, keepdim=True) / c["H"] if layer else torch.zeros(c["T"], 1, dtype=torch.float64, device=DEV)
        return mean, ((x - mean).pow(2).sum(-1, keepdim=True) / c["H"] + EPS).pow(-0.5)

    if op == "ln_fwd":
        x = st["x"] if st["residual"] is None else st["x"] + st["residual"]     # the stream keeps its own type
        mean, rstd = moments(x.double())
        out = {"y": norm(x.double(), f64(st["gamma"]), f64(st["beta"]), mean, rstd), "rstd": rstd[:, 0]}
        if layer:
            out["mean"] = mean[:, 0]
        if st["residual"] is not None:
            out["sum"] = st["x"].double() + st["residual"].double()
        return out
    if op == "ln_bwd":
        # the gradient of <dy, norm(x)>, a few thousand rows at a time
        gamma, beta = f64(st["gamma"]).requires_grad_(), f64(st["beta"]).requires_grad_()
        dx, step, T = [], 8192, c["T"]
        c = dict(c)
        for i in range(0, T, step):
            x = st["x"][i: i + step].double().requires_grad_()
            c["T"] = x.shape[0]
            (norm(x, gamma, beta, *moments(x)) * st["dy"][i: i + step].double()).sum().backward()
            dx.append(x.grad if st["dres"] is None else x.grad + st["dres"][i: i + step].double())
        out = {"dx": torch.cat(dx), "dgamma": gamma.grad}
        if layer:
            out["dbeta"] = beta.grad
        return out
    if op in ("router", "balance"):
        T, E, K = c["T"], c["E"], c["K"]
        seg = st["seg"].tolist()
        logits = st["logits"].double().requires_grad_()
        owner = torch.full((T,), len(seg) - 1, device=DEV)
        for i in range(len(seg) - 1):
            owner[seg[i]: seg[i + 1]] = i
        valid = owner < len(seg) - 1
        live = valid & (st["logits"] > NEG_INF).any(-1)
        rows = live.nonzero()[:, 0]
        logp = torch.log_softmax(logits[rows], -1)
        lse = torch.logsumexp(logits[rows], -1)
        prob = torch.zeros(len(seg), E, dtype=torch.float64, device=DEV).index_add(0, owner[rows], logp.exp())[:-1]
        length = torch.bincount(owner, minlength=len(seg))[:-1].double()
        n = max(1, int(length.sum()))
        key = torch.argsort(st["logits"][rows], dim=-1, descending=True, stable=True)[:, :K]
        chosen = torch.gather(logits[rows], 1, key)
        used = chosen > NEG_INF
        hits = torch.zeros(len(seg) * E, dtype=torch.float64, device=DEV)
        hits = hits.index_add(0, (owner[rows][:, None] * E + key)[used], torch.ones_like(chosen)[used])
        hits = hits.reshape(len(seg), E)[:-1]
        bal = ALPHA * sum((E * hits[i] / (K * length[i]) * prob[i] / length[i]).sum() * (length[i] / n)
                          for i in range(len(seg) - 1) if length[i] > 0)
        z = BETA * lse.square().sum() / n
        if op == "balance":
            total = bal * float(st["dloss"][0]) + z * float(st["dloss"][1])
            if not (torch.is_tensor(total) and total.requires_grad):
                return torch.zeros_like(logits) if st["add"] is None else st["add"].double()
            grad = torch.nan_to_num(torch.autograd.grad(total, logits)[0])
            return grad if st["add"] is None else grad + st["add"].double()
        scores = torch.zeros(T, K, dtype=torch.float64, device=DEV)
        sel = chosen if c["mode"] == 2 else torch.softmax(chosen, -1)
        if c["mode"] == 1 and not c["renorm"]:
            sel = torch.gather(logp, 1, key).exp()
        scores[rows] = torch.where(used, sel, torch.zeros_like(sel)).detach()
        every = torch.full((T,), NEG_INF, dtype=torch.float64, device=DEV)
        every[rows] = lse.detach()
        loss = torch.stack([torch.as_tensor(bal, device=DEV).detach().double(), z.detach()])
        return {"scores": scores, "ids": None, "lse": every, "counts": None, "prob_sum": prob.detach(), "loss": loss}
    if op == "pack":
        I, B = c["I"], c["B"]
        h = st["h"].double()
        a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        most = torch.zeros(st["N"] * B // 32, 2 * I, dtype=torch.float64, device=DEV)
        group = (st["slot"] // 32)[:, None].expand(-1, 2 * I)
        most = most.scatter_reduce(0, group, h.abs(), "amax")
        step = 2.0 ** (torch.floor(torch.log2(most.clamp(min=2.0 ** -120))) - 6)
        step = torch.gather(step, 0, group)
        return {"a": a, "h": torch.clamp(torch.round(h / step), -127, 127) * step}
    # the gradient of <dout, out> with the saved pre-activations in the place of x W1
    T, H, I, E, K, B = (c[k] for k in ("T", "H", "I", "E", "K", "B"))
    x, W1, W2, s = (st[k].double().requires_grad_() for k in ("x", "W1", "W2", "s"))
    total = 0.0
    sf = 2.0 ** (st["sf"].double() - 127)
    for e in range(E):
        mine = (st["expert"] == e).nonzero()[:, 0]
        if mine.numel() == 0:
            continue
        slot, flat = st["slot"][mine], st["order"][mine]
        b, j = slot // B, slot % B
        saved = st["q"].double()[b, :, :, j] * sf[b, :, j // 128, :, j % 128 // 32].reshape(-1, 2, I)
        xw = x[flat // K] @ W1[e]
        h = saved.reshape(-1, 2 * I) + (xw - xw.detach())
        y = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ W2[e]
        total = total + (s.flatten()[flat][:, None] * y * st["dout"].double()[flat // K]).sum()
    total.backward()
    return {"dx": x.grad, "dW1": W1.grad, "dW2": W2.grad, "ds": s.grad}


# ---------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        n, es = c["T"] * c["H"], 2 if c["type"] == "bf16" else 4
        if op == "ln_fwd":
            return {"bytes": n * es * (4 if c["skip"] else 2) + 8 * c["T"] + 8 * c["H"], "flops": 8 * n}
        return {"bytes": n * es * (4 if c["skip"] else 3) + 8 * c["T"] + 12 * c["H"], "flops": 14 * n}
    if op in ("router", "balance"):
        n = c["T"] * c["E"]
        table = 8 * c["S"] * c["E"]
        if op == "router":
            return {"bytes": 4 * n + 8 * c["T"] * c["K"] + 4 * c["T"] + table, "flops": 6 * n}
        return {"bytes": 4 * n * (3 if c["add"] else 2) + 4 * c["T"] + table // 2, "flops": 8 * n}
    rows = c["T"] * c["K"]
    if op == "pack":  # h read, a and the codes written; the codes read, the values written
        codes = 2 * c["I"] * rows * (1 + 1 / 32)
        return {"bytes": rows * c["I"] * 6 + 2 * codes + rows * c["I"] * 4, "flops": 20 * rows * c["I"]}
    T, H, I, E = c["T"], c["H"], c["I"], c["E"]
    return {"bytes": 6 * T * H + 12 * E * H * I + 2 * I * rows * (1 + 1 / 32) + 12 * rows, "flops": 12 * rows * H * I}
