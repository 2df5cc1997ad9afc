"""Measured cases of the dense branch beside the expert layer, in training, fine-tuning and serving.

  ffn_fwd / ffn_bwd          the gated feed-forward block (a shared expert): out = act(x Wg) * (x Wu) W2, and its
                             gradients from the saved pre-activations
  dropout                    dropout from a counter-based generator, with the residual add, and its gradient
  adapter_fwd / adapter_bwd  low-rank adapters of many requests added onto a projection's output, rows grouped by
                             route_meta, and their gradients

``run`` computes the plain form in elementary torch operations, or, where ``own`` is true, calls the
library.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # serving: one token through the fine-grained workload's shared expert, weights streamed once
        {"name": "ffn_fwd_token", "op": "ffn_fwd", "T": 1, "H": 2048, "I": 1024, "glu": 0, "interleaved": False, "bias": False, "save": False},
        # a ragged batch between serving and training: biases, interleaved columns, GELU, pre-activations kept
        {"name": "ffn_fwd_ragged", "op": "ffn_fwd", "T": 777, "H": 2048, "I": 768, "glu": 1, "interleaved": True, "bias": True, "save": True},
        # a training batch of the wide hidden size, pre-activations kept for the backward
        {"name": "ffn_fwd_large", "op": "ffn_fwd", "T": 16384, "H": 4096, "I": 2048, "glu": 0, "interleaved": False, "bias": False, "save": True},
        # gradients of a small odd block with its biases
        {"name": "ffn_bwd_small", "op": "ffn_bwd", "T": 333, "H": 520, "I": 264, "glu": 1, "interleaved": False, "bias": True},
        # gradients of that training batch
        {"name": "ffn_bwd_large", "op": "ffn_bwd", "T": 16384, "H": 4096, "I": 2048, "glu": 0, "interleaved": False, "bias": False},
        # dropout on the few rows of an interactive fine-tuning step: launch latency
        {"name": "dropout_few_rows", "op": "dropout", "T": 7, "H": 2048, "type": "bf16", "backward": False, "residual": True, "p": 0.1},
        # the branch's output dropped and added to the residual stream, the largest batch
        {"name": "dropout_large", "op": "dropout", "T": 65536, "H": 4096, "type": "bf16", "backward": False, "residual": True, "p": 0.1},
        # its gradient on an fp32 stream of odd width: rows that are not 16-byte aligned
        {"name": "dropout_bwd_odd", "op": "dropout", "T": 16411, "H": 1111, "type": "fp32", "backward": True, "residual": False, "p": 0.25},
        # serving: one new token for each of 48 requests, spread over 32 tenants' adapters
        {"name": "adapter_fwd_decode", "op": "adapter_fwd", "T": 48, "H": 4096, "N": 4096, "n": 32, "r": 16, "none": 0.0},
        # prefill of many requests on a few adapters, some requests without one
        {"name": "adapter_fwd_prefill", "op": "adapter_fwd", "T": 16384, "H": 4096, "N": 4096, "n": 8, "r": 16, "none": 0.1},
        # gradients on odd sizes and rank, some rows without an adapter
        {"name": "adapter_bwd_odd", "op": "adapter_bwd", "T": 513, "H": 1000, "N": 1240, "n": 5, "r": 12, "none": 0.2},
        # fine-tuning several tenants in one batch, rank 64
        {"name": "adapter_bwd_train", "op": "adapter_bwd", "T": 16384, "H": 4096, "N": 4096, "n": 4, "r": 64, "none": 0.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_bwd", "dropout", "adapter_fwd", "adapter_bwd"])
    if op in ("ffn_fwd", "ffn_bwd"):
        H, I = 8 * _log_int(rng, 8, 512), 8 * _log_int(rng, 8, 256)
        case = {"op": op, "T": _log_int(rng, 1, 16384), "H": H, "I": I, "glu": rng.randint(0, 1),
                "interleaved": rng.random() < 0.5, "bias": rng.random() < 0.5}
        return dict(case, save=rng.random() < 0.5) if op == "ffn_fwd" else case
    if op == "dropout":
        H = _log_int(rng, 16, 8192)
        if rng.random() < 0.5:
            H = -(-H // 64) * 64
        kind = rng.choice(["bf16", "fp32"])
        most = 65536 * 4096 // (2 if kind == "fp32" else 1) // H
        backward = rng.random() < 0.5
        return {"op": op, "T": _log_int(rng, 1, min(131072, most)), "H": H, "type": kind, "backward": backward,
                "residual": not backward and rng.random() < 0.6, "p": round(rng.uniform(0.02, 0.6), 3)}
    n = _log_int(rng, 1, 64)
    r = rng.choice([4, 8, 16, 32, 64, rng.randint(1, 64)])
    T = _log_int(rng, 1, 16384)
    if op == "adapter_bwd" and T * r > 16384 * 16:
        n = min(n, 16)
    return {"op": op, "T": T, "H": 8 * _log_int(rng, 8, 512), "N": 8 * _log_int(rng, 8, 512), "n": n, "r": r,
            "none": rng.choice([0.0, 0.1, 0.3])}


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------
def _rows_of_adapters(T, n, none, gen):
    """Adapter of each row (-1: none) as requests of uneven popularity bring it, and route_meta's grouping of the rows."""
    weight = 1.0 / torch.arange(1, n + 1, device=DEV, dtype=torch.float32)
    ids = torch.multinomial(weight, T, replacement=True, generator=gen)
    # consecutive rows belong to one request where there are many of them
    run = max(1, min(256, T // (2 * n)))
    ids = ids[torch.arange(T, device=DEV) // run]
    ids = torch.where((torch.rand(T, generator=gen, device=DEV) < none), torch.full_like(ids, -1), ids)
    have = ids >= 0
    order = torch.argsort(torch.where(have, ids, torch.full_like(ids, n)), stable=True)
    count = torch.bincount(ids[have], minlength=n)
    offsets = torch.cat([torch.zeros(1, device=DEV, dtype=torch.long), torch.cumsum(count, 0)])
    rows = int(offsets[-1])
    back = torch.full((T,), -1, device=DEV, dtype=torch.long)
    back[order[:rows]] = torch.arange(rows, device=DEV)
    gather = torch.full((T,), -1, device=DEV, dtype=torch.long)
    gather[:rows] = order[:rows]
    meta = {"expert_offsets": offsets.int(), "x_gather_idx": gather.int(), "s_reverse_scatter_idx": back.int()}
    return {"ids": ids, "route_meta": meta, "token": order[:rows], "expert": ids[order[:rows]],
            "place": torch.arange(rows, device=DEV) - offsets[ids[order[:rows]]], "capacity": max(1, int(count.max()))}


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    bf = torch.bfloat16
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if op in ("ffn_fwd", "ffn_bwd"):
        T, H, I = case["T"], case["H"], case["I"]
        st = {"x": rand(T, H).to(bf), "W1": (rand(H, 2 * I) * H ** -0.5).to(bf), "W2": (rand(I, H) * I ** -0.5).to(bf)}
        st["b1"] = (0.1 * rand(2 * I)).to(bf) if case["bias"] else None
        st["b2"] = (0.1 * rand(H)).to(bf) if case["bias"] else None
        if op == "ffn_bwd":
            h = st["x"] @ st["W1"]
            st["h"] = h + st["b1"] if case["bias"] else h
            st["dout"] = rand(T, H).to(bf)
    elif op == "dropout":
        T, H, dt = case["T"], case["H"], TYPES[case["type"]]
        st = {"x": rand(T, H).to(dt), "residual": rand(T, H).to(dt) if case["residual"] else None,
              "seed": 0x9D2C5680A7F1 + seed, "offset": (seed % 1000) << 30}
    else:
        T, H, N, n, r = (case[k] for k in ("T", "H", "N", "n", "r"))
        st = _rows_of_adapters(T, n, case["none"], gen)
        st.update(x=rand(T, H).to(bf), A=(rand(n, r, H) * H ** -0.5).to(bf), B=(rand(n, r, N) * r ** -0.5).to(bf),
                  scale=0.5 + torch.rand(n, generator=gen, device=DEV))
        if op == "adapter_fwd":
            st["base"] = rand(T, N).to(bf)
        else:
            st["dy"], st["base"] = rand(T, N).to(bf), rand(T, H).to(bf)
            st["u"] = _grouped(st, st["x"].float(), st["A"].float().transpose(1, 2))
    st["case"] = dict(case)
    return st


# ---------------------------------------------------------------------------------------------------
# plain forms: 32-bit torch operations
# ---------------------------------------------------------------------------------------------------
def _gate_up(h, c):
    return (h[:, 0::2], h[:, 1::2]) if c["interleaved"] else (h[:, : c["I"]], h[:, c["I"]:])


def _join(gate, up, c):
    return torch.stack([gate, up], 2).flatten(1) if c["interleaved"] else torch.cat([gate, up], 1)


def _activation(g, c):
    """act(g) and its derivative: SiLU, or GELU with the exact normal distribution."""
    if c["glu"] == 0:
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _plain_ffn_fwd(st, c):
    h = st["x"].float() @ st["W1"].float()
    if c["bias"]:
        h = h + st["b1"].float()
    gate, up = _gate_up(h, c)
    out = (_activation(gate, c)[0] * up) @ st["W2"].float()
    if c["bias"]:
        out = out + st["b2"].float()
    out = {"out": out.to(torch.bfloat16)}
    if c["save"]:
        out["h"] = h.to(torch.bfloat16)
    return out


def _plain_ffn_bwd(st, c):
    x, dout, W1, W2 = (st[k].float() for k in ("x", "dout", "W1", "W2"))
    gate, up = _gate_up(st["h"].float(), c)
    act, slope = _activation(gate, c)
    da = dout @ W2.t()
    dh = _join(da * up * slope, da * act, c)
    bf = torch.bfloat16
    out = {"dx": (dh @ W1.t()).to(bf), "dW1": (x.t() @ dh).to(bf), "dW2": ((act * up).t() @ dout).to(bf)}
    if c["bias"]:
        out["db1"], out["db2"] = dh.double().sum(0).float(), dout.double().sum(0).float()
    return out


LOW = 0xFFFFFFFF


def _keep(c, seed, offset):
    """[T, H] truth values: Philox4x32-10 (Salmon et al. 2011) with the key `seed` on the counter (column / 4, row,
    offset); word column % 4 is at least p 2^32."""
    T, H = c["T"], c["H"]
    quads = -(-H // 4)
    x0 = torch.arange(quads, device=DEV).expand(T, quads)
    x1 = torch.arange(T, device=DEV)[:, None].expand(T, quads)
    x2, x3 = torch.full_like(x0, offset & LOW), torch.full_like(x0, offset >> 32)
    k0, k1 = seed & LOW, seed >> 32
    for i in range(10):
        p0, p1 = x0 * 0xD2511F53, x2 * 0xCD9E8D57      # 64-bit products; their sign does not matter to the halves
        x0 = ((p1 >> 32) & LOW) ^ x1 ^ ((k0 + i * 0x9E3779B9) & LOW)
        x2 = ((p0 >> 32) & LOW) ^ x3 ^ ((k1 + i * 0xBB67AE85) & LOW)
        x1, x3 = p1 & LOW, p0 & LOW
    words = torch.stack([x0, x1, x2, x3], 2).reshape(T, -1)[:, :H]
    return words >= int(c["p"] * 2.0 ** 32 + 0.5)


def _plain_dropout(st, c):
    y = st["x"].float() * (1 / (1 - c["p"]))
    y = torch.where(_keep(c, st["seed"], st["offset"]), y, torch.zeros_like(y))
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(st["x"].dtype)


def _padded(st, rows):
    """Grouped rows, padded to the same number for every adapter: [n, capacity, columns]."""
    n, cap = st["A"].shape[0], st["capacity"]
    out = torch.zeros(n * cap, rows.shape[1], device=DEV, dtype=rows.dtype)
    return out.index_copy_(0, st["expert"] * cap + st["place"], rows).reshape(n, cap, -1)


def _grouped(st, rows, weights):
    """rows [T, K] times each row's own weights [n, K, M]; zeros for rows without an adapter."""
    cap = st["capacity"]
    prod = torch.bmm(_padded(st, rows[st["token"]]), weights).reshape(-1, weights.shape[2])
    out = torch.zeros(rows.shape[0], weights.shape[2], device=DEV, dtype=rows.dtype)
    return out.index_copy_(0, st["token"], prod[st["expert"] * cap + st["place"]])


def _row_scale(st):
    return torch.where(st["ids"] >= 0, st["scale"][st["ids"].clamp(min=0)], torch.zeros_like(st["scale"][:1]))[:, None]


def _plain_adapter_fwd(st, c):
    u = _grouped(st, st["x"].float(), st["A"].float().transpose(1, 2))
    y = st["base"].float() + _grouped(st, u * _row_scale(st), st["B"].float())
    return {"y": y.to(torch.bfloat16), "u": u}


def _plain_adapter_bwd(st, c):
    dy, x, A, B = (st[k].float() for k in ("dy", "x", "A", "B"))
    scale = _row_scale(st)
    v = _grouped(st, dy, B.transpose(1, 2)) * scale
    dx = st["base"].float() + _grouped(st, v, A)
    group = lambda t: _padded(st, t[st["token"]])  # noqa: E731
    dA = torch.bmm(group(v).transpose(1, 2), group(x))
    dB = torch.bmm(group(st["u"] * scale).transpose(1, 2), group(dy))
    bf = torch.bfloat16
    return {"dx": dx.to(bf), "dA": dA.to(bf), "dB": dB.to(bf)}


PLAIN = {"ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd, "dropout": _plain_dropout, "adapter_fwd": _plain_adapter_fwd,
         "adapter_bwd": _plain_adapter_bwd}


# ---------------------------------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------------------------------
def _own(st, c):
    import moe_expert_layer_routing_gb300 as mb
    op = c["op"]
    if op in ("ffn_fwd", "ffn_bwd"):
        how = dict(glu=mb.GLU_GEGLU if c["glu"] else mb.GLU_SWIGLU,
                   gate_up_layout=mb.GATE_UP_INTERLEAVED if c["interleaved"] else mb.GATE_UP_CONCAT)
        if op == "ffn_fwd":
            r = mb.ffn_fwd(st["x"], st["W1"], st["W2"], b1=st["b1"], b2=st["b2"], save=c["save"], **how)
            return {k: r[k] for k in ["out"] + ["h"] * c["save"]}
        r = mb.ffn_bwd(st["dout"], st["x"], st["h"], st["W1"], st["W2"], bias=c["bias"], **how)
        return {k: r[k] for k in ["dx", "dW1", "dW2"] + ["db1", "db2"] * c["bias"]}
    if op == "dropout":
        if c["backward"]:
            return mb.dropout_bwd(st["x"], c["p"], st["seed"], st["offset"])
        return mb.dropout_fwd(st["x"], c["p"], st["seed"], st["offset"], residual=st["residual"])
    if op == "adapter_fwd":
        r = mb.adapter_fwd(st["x"], st["A"], st["B"], st["route_meta"], scale=st["scale"], base=st["base"])
        return {k: r[k] for k in ("y", "u")}
    r = mb.adapter_bwd(st["dy"], st["x"], st["u"], st["A"], st["B"], st["route_meta"], scale=st["scale"], base=st["base"])
    return {k: r[k] for k in ("dx", "dA", "dB")}


def run(state):
    c = state["case"]
    return _own(state, c) if own else PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------------------------------
def _exact_words(rows, cols, seed, offset):
    """The four words of the generator for these rows and column quads, products from 16-bit limbs."""
    def product(a, m):
        lo, hi = a & 0xFFFF, a >> 16
        m0, m1 = m & 0xFFFF, m >> 16
        mid = hi * m0 + ((lo * m0) >> 16)
        mid2 = lo * m1 + (mid & 0xFFFF)
        return hi * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((lo * m0) & 0xFFFF)

    shape = (rows.numel(), cols.numel())
    w = [cols[None].expand(shape), rows[:, None].expand(shape), torch.full(shape, offset % 2 ** 32, device=DEV),
         torch.full(shape, offset // 2 ** 32, device=DEV)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = product(w[0], 0xD2511F53)
        h1, l1 = product(w[2], 0xCD9E8D57)
        w = [h1 ^ w[1] ^ key[0], l1, h0 ^ w[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return w


def exact(case, seed):
    st, c, op = prepare(case, seed), case, case["op"]
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    act = torch.nn.functional.silu if c.get("glu") == 0 else torch.nn.functional.gelu
    if op in ("ffn_fwd", "ffn_bwd"):
        x, W1, W2 = (f64(st[k]) for k in ("x", "W1", "W2"))
        pick = (lambda h: (h[:, 0::2], h[:, 1::2])) if c["interleaved"] else (lambda h: h.chunk(2, 1))
    if op == "ffn_fwd":
        h = x @ W1 if st["b1"] is None else torch.addmm(f64(st["b1"]), x, W1)
        gate, up = pick(h)
        out = (act(gate) * up) @ W2
        out = {"out": out if st["b2"] is None else out + f64(st["b2"])}
        return dict(out, h=h) if c["save"] else out
    if op == "ffn_bwd":
        # the gradient of <dout, out> by the saved pre-activations, and from there through h = x W1 + b1
        h, W2 = f64(st["h"]).requires_grad_(), W2.requires_grad_()
        gate, up = pick(h)
        ((act(gate) * up @ W2) * f64(st["dout"])).sum().backward()
        out = {"dx": h.grad @ W1.mT, "dW1": x.mT @ h.grad, "dW2": W2.grad}
        return dict(out, db1=h.grad.sum(0), db2=f64(st["dout"]).sum(0)) if c["bias"] else out
    if op == "dropout":
        T, H = c["T"], c["H"]
        y = torch.empty(T, H, dtype=torch.float64, device=DEV)
        cols = torch.arange((H + 3) // 4, device=DEV)
        border = int(c["p"] * 2.0 ** 32 + 0.5)
        for i in range(0, T, 8192):
            rows = torch.arange(i, min(T, i + 8192), device=DEV)
            words = _exact_words(rows, cols, st["seed"], st["offset"])
            for k in range(4):
                mine = slice(k, None, 4)
                part = f64(st["x"][i: i + 8192, mine]) / (1 - c["p"])
                y[i: i + 8192, mine] = part * (words[k][:, : part.shape[1]] >= border)
        return y if st["residual"] is None else y + f64(st["residual"])
    # adapter by adapter
    x, A, B, base, scale = (f64(st[k]) for k in ("x", "A", "B", "base", "scale"))
    out = {"y": base.clone(), "u": torch.zeros(c["T"], c["r"], dtype=torch.float64, device=DEV)} if op == "adapter_fwd" else \
        {"dx": base.clone(), "dA": torch.zeros_like(A), "dB": torch.zeros_like(B)}
    for a in range(c["n"]):
        rows = (st["ids"] == a).nonzero()[:, 0]
        if op == "adapter_fwd":
            u = x[rows] @ A[a].mT
            out["u"][rows] = u
            out["y"][rows] += scale[a] * (u @ B[a])
        else:
            dy, u = f64(st["dy"][rows]), f64(st["u"][rows])
            v = scale[a] * (dy @ B[a].mT)
            out["dx"][rows] += v @ A[a]
            out["dA"][a] = v.mT @ x[rows]
            out["dB"][a] = scale[a] * (u.mT @ dy)
    return out


# ---------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    if op in ("ffn_fwd", "ffn_bwd"):
        T, H, I = c["T"], c["H"], c["I"]
        weights = 3 * H * I
        if op == "ffn_fwd":
            return {"bytes": 2 * (2 * T * H + weights + (2 * T * I if c["save"] else 0)), "flops": 6 * T * H * I}
        return {"bytes": 2 * (3 * T * H + 2 * T * I + 2 * weights), "flops": 12 * T * H * I}
    if op == "dropout":
        n = c["T"] * c["H"]
        return {"bytes": n * (2 if c["type"] == "bf16" else 4) * (3 if c["residual"] else 2), "flops": 40 * n}
    T, H, N, n, r = (c[k] for k in ("T", "H", "N", "n", "r"))
    n = min(n, T)       # adapters that a row can name
    if op == "adapter_fwd":
        return {"bytes": 2 * T * H + 4 * T * N + 2 * n * r * (H + N) + 4 * T * r, "flops": 2 * T * r * (H + N)}
    return {"bytes": 2 * T * N + 6 * T * H + 4 * n * r * (H + N) + 4 * T * r, "flops": 4 * T * r * (H + N)}
