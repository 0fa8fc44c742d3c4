"""Cases of the operators between the token ids and the FP8 products: layer
norm, dropout, the router of a mixture-of-experts block, the embedding.

``run`` computes a case in plain torch operations (32-bit arithmetic, one
rounding at the end), or, with ``own`` true, through the library's entry
points.  ``exact`` computes the same from the definitions in 64 bits.

Notation: T tokens, H hidden size, E experts, K experts per token, V rows of
the embedding table.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 0), "e5m2": (torch.float8_e5m2, 57344.0, 1)}
EPS = 1e-5
BALANCE, Z = 1e-2, 1e-3
LOW32 = 0xFFFFFFFF
# Philox4x32: the multipliers of a round, and what is added to the key after it
MULTIPLIERS, KEY_STEPS, ROUNDS = (0xD2511F53, 0xCD9E8D57), (0x9E3779B9, 0xBB67AE85), 10


# ---------------------------------------------------------------- the cases
def listed():
    def norm(name, op, rows, hidden, **more):
        return {"name": name, "op": op, "rows": rows, "hidden": hidden, "dtype": "bf16",
                "res": "bf16", "param": "bf16", "offset": 0.0, "p": 0.1, "site": 3, "fp8": "none",
                **more}

    def drop(name, rows, hidden, **more):
        return {"name": name, "op": "dropout", "rows": rows, "hidden": hidden, "dtype": "bf16",
                "p": 0.1, "site": 0, **more}

    def route(name, op, tokens, experts, topk, **more):
        return {"name": name, "op": op, "tokens": tokens, "experts": experts, "topk": topk,
                "dtype": "fp32", "normalize": True, "masked": True, **more}

    def embed(name, op, tokens, vocab, hidden, **more):
        return {"name": name, "op": op, "tokens": tokens, "vocab": vocab, "hidden": hidden,
                "dtype": "bf16", "grad": "fp32", "index": "int64", **more}

    return [
        # one decoding step: the residual sum and the norm that feeds an FP8 product, nothing dropped
        norm("layer norm decode fp8", "norm", 4, 4096, p=0.0, fp8="e4m3"),
        # a training micro-batch with an odd token count
        norm("layer norm train", "norm", 8191, 6144),
        # odd hidden size, half precision around an fp32 residual stream, weights kept as w - 1
        norm("layer norm backward odd", "norm_bwd", 4099, 777, dtype="fp16", res="fp32",
             param="fp32", offset=1.0),
        # the largest training junction
        norm("layer norm backward train", "norm_bwd", 8192, 12288),
        # the branch of a short fine-tuning micro-batch
        drop("dropout small", 64, 4096),
        # behind the embedding of a large batch, rows that are not whole 16-byte blocks
        drop("dropout train odd", 8191, 12287),
        # one decoding step through a router
        route("router decode", "router", 4, 64, 4, masked=False),
        # a training micro-batch, many experts
        route("router train", "router", 16384, 256, 8),
        # its gradient, logits of half the width, probabilities over all experts
        route("router backward train", "router_bwd", 8191, 64, 4, dtype="bf16", normalize=False),
        # a training micro-batch of ids
        embed("embedding train", "embedding", 16384, 65536, 6144),
        # the gradient of a short micro-batch into a small table
        embed("embedding backward small", "embedding_bwd", 1000, 2000, 512, grad="bf16",
              index="int32"),
        # the gradient of a training micro-batch, fp32 for the optimizer
        embed("embedding backward train", "embedding_bwd", 16384, 65536, 4096),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _hidden(rng, lo, hi):
    """Half of the draws a multiple of 64, the rest of 8 or any number."""
    h = _log_int(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    return max(step, h // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "dropout", "router", "router_bwd", "embedding",
                     "embedding_bwd"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op in ("norm", "norm_bwd"):
        case = {"op": op, "rows": _log_int(rng, 1, 16384), "hidden": _hidden(rng, 512, 12288),
                "dtype": dtype, "res": rng.choice((dtype, "fp32")),
                "param": rng.choice((dtype, "fp32")), "offset": rng.choice((0.0, 1.0)),
                "p": rng.choice((0.0, 0.05, 0.1, 0.5)), "site": rng.randint(0, 500),
                "fp8": rng.choice(("none", "none", "e4m3", "e5m2")) if op == "norm" else "none"}
        rows = "rows"
    elif op == "dropout":
        case = {"op": op, "rows": _log_int(rng, 1, 16384), "hidden": _hidden(rng, 512, 12288),
                "dtype": dtype, "p": rng.choice((0.05, 0.1, 0.5)), "site": rng.randint(0, 500)}
        rows = "rows"
    elif op in ("router", "router_bwd"):
        experts = _log_int(rng, 8, 256)
        case = {"op": op, "tokens": _log_int(rng, 1, 32768), "experts": experts,
                "topk": rng.randint(1, 8), "dtype": rng.choice(("fp32", "fp32", "bf16", "fp16")),
                "normalize": rng.random() < 0.5, "masked": rng.random() < 0.5}
        rows = "tokens"
    else:
        case = {"op": op, "tokens": _log_int(rng, 1, 32768), "vocab": _log_int(rng, 1000, 131072),
                "hidden": _hidden(rng, 512, 12288), "dtype": dtype,
                "grad": rng.choice((dtype, "fp32")), "index": rng.choice(("int32", "int64"))}
        while case["vocab"] * case["hidden"] > 2.2e8:
            case["vocab"] = case["vocab"] * 3 // 4
        rows = "tokens"
    while work(case)["bytes"] > 1.1e9 and case[rows] > 1:
        case[rows] = case[rows] * 3 // 4
    return case


def _distinct(tokens, vocab):
    """Expected number of different ids among the tokens (see _ids)."""
    edge = torch.log(torch.arange(1, vocab + 2, dtype=torch.float64))
    share = (edge[1:] - edge[:-1]) / edge[-1]
    return int((1 - (1 - share) ** tokens).sum())


def work(c):
    if c["op"] in ("norm", "norm_bwd"):
        x, r, t = SIZE[c["dtype"]], SIZE[c["res"]], c["rows"] * c["hidden"]
        if c["op"] == "norm":
            return {"bytes": t * (x + 2 * r + (x if c["fp8"] == "none" else 1)) + 8 * c["rows"],
                    "flops": 12 * t}
        return {"bytes": t * (2 * x + 3 * r) + 8 * c["rows"], "flops": 16 * t}
    if c["op"] == "dropout":
        t = c["rows"] * c["hidden"]
        return {"bytes": 2 * SIZE[c["dtype"]] * t, "flops": 2 * t}
    if c["op"] in ("router", "router_bwd"):
        t, one = c["tokens"], c["tokens"] * c["experts"]
        sides = 1 if c["op"] == "router" else 2
        return {"bytes": sides * SIZE[c["dtype"]] * one + 8 * t * c["topk"] + t
                + 4 * c["experts"], "flops": 8 * one}
    t, h, i = c["tokens"], c["hidden"], 4 if c["index"] == "int32" else 8
    b = SIZE[c["dtype"]]
    if c["op"] == "embedding":
        return {"bytes": b * h * (t + _distinct(t, c["vocab"])) + i * t, "flops": t * h}
    return {"bytes": b * h * t + SIZE[c["grad"]] * c["vocab"] * h + i * t, "flops": t * h}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"n": _prepare_norm, "d": _prepare_dropout, "r": _prepare_router,
            "e": _prepare_embedding}[case["op"][0]]
    return make(dict(case), g)


def _normal(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _empty(*shape, dtype=torch.float32):
    return torch.empty(*shape, device="cuda", dtype=dtype)


def _random_state(g):
    """Seed and step of the generator, as a training program keeps them."""
    return torch.randint(0, 2 ** 62, (2,), generator=g, device="cuda")


def _prepare_norm(c, g):
    rows, h = c["rows"], c["hidden"]
    x, r, p = DTYPES[c["dtype"]], DTYPES[c["res"]], DTYPES[c["param"]]
    s = {"case": c, "rng": _random_state(g),
         "weight": _normal(g, h, std=0.2).add_(1 - c["offset"]).to(p),
         "bias": _normal(g, h, std=0.2, dtype=p)}
    # a residual stream whose channels have means of their own
    stream = _normal(g, rows, h, std=2.0).add_(_normal(g, h, std=0.5)).add_(0.5)
    if c["op"] == "norm":
        s["u"], s["res"] = _normal(g, rows, h, std=0.7, dtype=x), stream.to(r)
        s["res_out"] = torch.empty_like(s["res"])
        s["mean"], s["rstd"] = _empty(rows), _empty(rows)
        s["y"] = _empty(rows, h, dtype=x if c["fp8"] == "none" else torch.uint8)
        if c["fp8"] != "none":  # a delayed scale: from an earlier step's largest output
            s["scale"] = torch.full((1,), FP8[c["fp8"]][1] / 7.0, device="cuda")
            s["amax"], s["scale_inv"] = (torch.zeros(1, device="cuda") for _ in range(2))
        return s
    # what the forward pass has kept, and the two gradients that come back
    s["res_out"] = stream.to(r)
    var, mean = torch.var_mean(s["res_out"].double(), 1, correction=0)
    s["mean"], s["rstd"] = mean.float(), torch.rsqrt(var + EPS).float()
    s["dy"] = _normal(g, rows, h, std=0.05, dtype=x)
    s["dres_out"] = _normal(g, rows, h, std=0.05, dtype=r)
    s["dres"], s["du"] = torch.empty_like(s["res_out"]), torch.empty_like(s["dy"])
    s["dweight"], s["dbias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
    return s


def _prepare_dropout(c, g):
    x = _normal(g, c["rows"], c["hidden"], dtype=DTYPES[c["dtype"]])
    return {"case": c, "x": x, "out": torch.empty_like(x), "rng": _random_state(g)}


def _prepare_router(c, g):
    t, e, k = c["tokens"], c["experts"], min(c["topk"], c["experts"])
    # a router that prefers some experts
    logits = _normal(g, t, e).add_(_normal(g, 1, e, std=0.8)).to(DTYPES[c["dtype"]])
    mask = None
    if c["masked"]:  # one token in 50 is padding
        mask = torch.rand(t, generator=g, device="cuda") >= 0.02
        mask[0] = True
    s = {"case": c, "topk": k, "logits": logits, "mask": mask}
    if c["op"] == "router":
        s.update(idx=_empty(t, k, dtype=torch.int32), weights=_empty(t, k),
                 counts=_empty(e + 1, dtype=torch.int32), loss=_empty(1))
        return s
    s["idx"], s["counts"] = _plain_choice(logits, mask, k)[:2]
    s["dweights"] = _normal(g, t, k, std=0.05)
    s["dloss"] = torch.full((1,), 0.5, device="cuda")
    s["dlogits"] = torch.empty_like(logits)
    return s


def _ids(c, g):
    """Ids of text, low ones frequent: the logarithm of id + 1 is uniform.
    One position in 100 is padding."""
    u = torch.rand(c["tokens"], generator=g, device="cuda", dtype=torch.float64)
    ids = torch.exp(u * math.log(c["vocab"] + 1)).long() - 1
    ids = ids.clamp_(0, c["vocab"] - 1)
    pad = torch.rand(c["tokens"], generator=g, device="cuda") < 0.01
    return torch.where(pad, -1, ids).to(getattr(torch, c["index"]))


def _prepare_embedding(c, g):
    t, v, h, x = c["tokens"], c["vocab"], c["hidden"], DTYPES[c["dtype"]]
    s = {"case": c, "idx": _ids(c, g), "scale": math.sqrt(h)}
    if c["op"] == "embedding":
        s["table"] = _normal(g, v, h, std=0.02, dtype=x)
        s["out"] = _empty(t, h, dtype=x)
        return s
    s["dout"] = _normal(g, t, h, std=0.05, dtype=x)
    s["dtable"] = _empty(v, h, dtype=DTYPES[c["grad"]])
    return s


# ---------------------------------------------------------------- plain forms
def _threshold(p):
    return int(p * 65536 + 0.5)


def _plain_keep(rows, hidden, p, rng, site):
    """Which elements stay: 16 bits of Philox4x32-10 each, eight columns of a
    row to a call.  Products wrap at 64 bits, as they should."""
    w = [torch.arange(-(-hidden // 8), device="cuda")[None, :].expand(rows, -1),
         torch.arange(rows, device="cuda")[:, None].expand(-1, -(-hidden // 8)),
         torch.full((1, 1), site, device="cuda"), (rng[1] & LOW32).view(1, 1)]
    key = [rng[0] & LOW32, (rng[0] >> 32) & LOW32]
    for _ in range(ROUNDS):
        a, b = w[0] * MULTIPLIERS[0], w[2] * MULTIPLIERS[1]
        w = [((b >> 32) & LOW32) ^ w[1] ^ key[0], b & LOW32,
             ((a >> 32) & LOW32) ^ w[3] ^ key[1], a & LOW32]
        key = [(k + step) & LOW32 for k, step in zip(key, KEY_STEPS)]
    bits = torch.stack([h for v in w for h in (v & 0xFFFF, v >> 16)], 2)
    return bits.view(rows, -1)[:, :hidden] >= _threshold(p)


def _plain_dropped(x, c, rng):
    if _threshold(c["p"]) == 0:
        return x
    keep = _plain_keep(*x.shape, c["p"], rng, c["site"])
    return torch.where(keep, x * (65536 / (65536 - _threshold(c["p"]))), 0.0)


def _plain_norm(s):
    c = s["case"]
    w = s["weight"].float() + c["offset"]
    if c["op"] == "norm":
        v = s["res"].float() + _plain_dropped(s["u"].float(), c, s["rng"])
        mean = v.mean(1)
        away = v - mean[:, None]
        rstd = torch.rsqrt((away * away).mean(1) + EPS)
        y = away * rstd[:, None] * w + s["bias"].float()
        out = {"res_out": v.to(s["res"].dtype), "mean": mean, "rstd": rstd}
        if c["fp8"] == "none":
            return {"y": y.to(s["u"].dtype), **out}
        dtype, top, _ = FP8[c["fp8"]]
        return {"y": (y * s["scale"]).clamp(-top, top).to(dtype),
                "amax": torch.maximum(s["amax"], y.abs().max()), "scale_inv": 1.0 / s["scale"],
                **out}
    dy = s["dy"].float()
    hat = (s["res_out"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    back = dy * w
    dres = s["dres_out"].float() + s["rstd"][:, None] * (
        back - back.mean(1, keepdim=True) - hat * (back * hat).mean(1, keepdim=True))
    return {"dres": dres.to(s["dres"].dtype),
            "du": _plain_dropped(dres, c, s["rng"]).to(s["du"].dtype),
            "dweight": (dy * hat).sum(0).to(s["weight"].dtype),
            "dbias": dy.sum(0).to(s["bias"].dtype)}


def _plain_choice(logits, mask, k):
    """Experts of every token, the slots per expert and (last) the number of
    tokens, and which tokens count."""
    t, e = logits.shape
    best, idx = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    valid = best[:, 0] > -math.inf if mask is None else mask & (best[:, 0] > -math.inf)
    idx = torch.where(valid[:, None] & (best[:, :k] > -math.inf), idx[:, :k], -1)
    hot = torch.zeros(e + 1, dtype=torch.int32, device=logits.device)
    hot.scatter_add_(0, torch.where(idx < 0, e, idx).view(-1),
                     torch.ones(t * k, dtype=torch.int32, device=logits.device))
    hot[e] = valid.sum()
    return idx.to(torch.int32), hot, valid


def _plain_router(s):
    c = s["case"]
    e, k = c["experts"], s["topk"]
    x = s["logits"].float()
    if c["op"] == "router":
        idx, counts, valid = _plain_choice(s["logits"], s["mask"], k)
    else:
        idx, counts = s["idx"], s["counts"]
        valid = x.amax(1) > -math.inf if s["mask"] is None else s["mask"]
    x = torch.where(valid[:, None], x, 0.0)
    top = x.amax(1, keepdim=True)
    part = torch.exp(x - top)
    total = part.sum(1, keepdim=True)
    p, lse = part / total, (top + torch.log(total))[:, 0]
    n = counts[e].clamp(min=1)
    load = counts[:e] / (n * k)
    chosen, at = idx >= 0, idx.long().clamp(min=0)
    weights = torch.where(chosen, p.gather(1, at), 0.0)
    sums = weights.sum(1, keepdim=True) if c["normalize"] else 1.0
    weights = torch.where(chosen, weights / sums, 0.0)
    if c["op"] == "router":
        mean = torch.where(valid[:, None], p, 0.0).sum(0) / n
        loss = BALANCE * e * (load * mean).sum() + Z * torch.where(valid, lse * lse, 0.0).sum() / n
        return {"idx": idx, "weights": weights, "counts": counts, "loss": loss.view(1)}
    dw = torch.where(chosen, s["dweights"], 0.0)
    each = (s["dloss"] * BALANCE * e / n) * load.expand_as(p)
    if not c["normalize"]:
        each = each.scatter_add(1, at, dw)
    dl = p * (each - (p * each).sum(1, keepdim=True))
    if c["normalize"]:
        dl = dl.scatter_add(1, at, weights * (dw - (weights * dw).sum(1, keepdim=True)))
    dl = dl + p * (2 * Z * s["dloss"] / n * lse[:, None])
    return torch.where(valid[:, None], dl, 0.0).to(s["logits"].dtype)


def _plain_embedding(s):
    v = s["case"]["vocab"]
    idx = s["idx"].long()
    here = ((idx >= 0) & (idx < v))[:, None]
    if s["case"]["op"] == "embedding":
        rows = s["table"][idx.clamp(0, v - 1)].float() * s["scale"]
        return torch.where(here, rows, 0.0).to(s["table"].dtype)
    total = torch.zeros(s["dtable"].shape, device="cuda")
    total.index_add_(0, idx.clamp(0, v - 1), torch.where(here, s["dout"].float(), 0.0))
    return (total * s["scale"]).to(s["dtable"].dtype)


# ---------------------------------------------------------------- the library
def _own_norm(s):
    import cast_transpose_gb300 as ct
    c = s["case"]
    same = {"weight": s["weight"], "weight_offset": c["offset"], "p": c["p"], "rng": s["rng"],
            "site": c["site"], "mean": s["mean"], "rstd": s["rstd"]}
    if c["op"] == "norm":
        out = {"res_out": s["res_out"], "mean": s["mean"], "rstd": s["rstd"]}
        if c["fp8"] == "none":
            ct.layer_norm(s["u"], s["res"], s["res_out"], s["y"], bias=s["bias"], eps=EPS, **same)
            return {"y": s["y"], **out}
        dtype, _, fmt = FP8[c["fp8"]]
        ct.layer_norm(s["u"], s["res"], s["res_out"], s["y"], bias=s["bias"], eps=EPS,
                      scale=s["scale"], amax=s["amax"], scale_inv=s["scale_inv"], fmt=fmt, **same)
        return {"y": s["y"].view(dtype), "amax": s["amax"], "scale_inv": s["scale_inv"], **out}
    if "workspace" not in s:
        size = ct.layer_norm_backward_workspace_size(c["rows"], c["hidden"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = {k: s[k] for k in ("dres", "du", "dweight", "dbias")}
    ct.layer_norm_backward(s["dy"], s["dres_out"], s["res_out"], workspace=s["workspace"],
                           **same, **out)
    return out


def _own_router(s):
    import cast_transpose_gb300 as ct
    c = s["case"]
    same = {"mask": s["mask"], "normalize": c["normalize"], "balance": BALANCE, "z": Z}
    if c["op"] == "router":
        if "workspace" not in s:
            size = ct.moe_router_workspace_size(c["tokens"], s["topk"], c["experts"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        out = {k: s[k] for k in ("idx", "weights", "counts", "loss")}
        ct.moe_router(s["logits"], s["idx"], s["weights"], s["counts"], s["loss"],
                      workspace=s["workspace"], **same)
        return out
    ct.moe_router_backward(s["dweights"], s["dloss"], s["logits"], s["idx"], s["counts"],
                           s["dlogits"], **same)
    return s["dlogits"]


def _own_embedding(s):
    import cast_transpose_gb300 as ct
    c = s["case"]
    if c["op"] == "embedding":
        ct.embedding(s["idx"], s["table"], s["out"], scale=s["scale"])
        return s["out"]
    if "workspace" not in s:
        size = ct.embedding_backward_workspace_size(c["tokens"], c["vocab"], c["hidden"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    ct.embedding_backward(s["idx"], s["dout"], s["dtable"], s["workspace"], scale=s["scale"])
    return s["dtable"]


def _own_dropout(s):
    import cast_transpose_gb300 as ct
    ct.dropout(s["x"], s["out"], s["case"]["p"], s["rng"], s["case"]["site"])
    return s["out"]


def run(state):
    kind = state["case"]["op"][0]
    if own:
        return {"n": _own_norm, "d": _own_dropout, "r": _own_router, "e": _own_embedding}[kind](state)
    if kind == "d":
        x = state["x"]
        return _plain_dropped(x.float(), state["case"], state["rng"]).to(x.dtype)
    return {"n": _plain_norm, "r": _plain_router, "e": _plain_embedding}[kind](state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["op"][0]
    if kind == "d":
        return s["x"].double() * _exact_factor(case, s["rng"], *s["x"].shape)
    return {"n": _exact_norm, "r": _exact_router, "e": _exact_embedding}[kind](s)


def _high_product(a, b):
    """The upper 32 bits of products of 32-bit numbers, from 16-bit halves."""
    a1, a0, b1, b0 = a // 65536, a % 65536, b // 65536, b % 65536
    low = a0 * b0
    mid = a1 * b0 + low // 65536
    return a1 * b1 + mid // 65536 + (a0 * b1 + mid % 65536) // 65536


def _exact_factor(c, rng, rows, hidden):
    """What dropout multiplies every element by, some rows at a time."""
    cut = _threshold(c["p"])
    if cut == 0:
        return 1.0
    seed, step = (int(v) for v in rng.tolist())
    groups = (hidden + 7) // 8
    factor = torch.empty(rows, hidden, dtype=torch.float64, device="cuda")
    for r0 in range(0, rows, 1024):
        r1 = min(rows, r0 + 1024)
        zero = torch.zeros(r1 - r0, groups, dtype=torch.long, device="cuda")
        x0 = zero + torch.arange(groups, device="cuda")
        x1 = zero + torch.arange(r0, r1, device="cuda")[:, None]
        x2, x3 = zero + c["site"], zero + step % 2 ** 32
        for i in range(ROUNDS):
            k0 = (seed + i * KEY_STEPS[0]) % 2 ** 32
            k1 = (seed // 2 ** 32 + i * KEY_STEPS[1]) % 2 ** 32
            m0, m1 = MULTIPLIERS
            x0, x1, x2, x3 = (_high_product(x2, m1) ^ x1 ^ k0, x2 * (m1 % 65536) % 2 ** 32
                              + x2 % 65536 * (m1 // 65536) * 65536 % 2 ** 32,
                              _high_product(x0, m0) ^ x3 ^ k1, x0 * (m0 % 65536) % 2 ** 32
                              + x0 % 65536 * (m0 // 65536) * 65536 % 2 ** 32)
            x1, x3 = x1 % 2 ** 32, x3 % 2 ** 32
        for j, word in enumerate((x0, x1, x2, x3)):
            for half, bits in enumerate((word % 65536, word // 65536)):
                at = factor[r0:r1, 2 * j + half::8]
                at.copy_((bits[:, :at.shape[1]] >= cut) * (65536 / (65536 - cut)))
    return factor


def _exact_norm(s):
    c = s["case"]
    w, h = s["weight"].double() + c["offset"], c["hidden"]
    if c["op"] == "norm":
        v = s["u"].double() * _exact_factor(c, s["rng"], *s["u"].shape) + s["res"].double()
        var, mean = torch.var_mean(v, 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["bias"].double(), v - mean[:, None], rstd[:, None] * w)
        out = {"res_out": v, "mean": mean, "rstd": rstd}
        if c["fp8"] == "none":
            return {"y": y, **out}
        dtype, top, _ = FP8[c["fp8"]]
        q = (y * s["scale"].double()).clamp(-top, top).to(dtype).double()
        return {"y": q, "amax": y.abs().max().reshape(1), "scale_inv": 1 / s["scale"].double(),
                **out}
    # from the Jacobian: J v = rstd (v - 1 (1 . v) / H - hat (hat . v) / H)
    dy, rstd = s["dy"].double(), s["rstd"].double()
    hat = torch.einsum("rh,r->rh", s["res_out"].double() - s["mean"].double()[:, None], rstd)
    v = dy * w
    along, level = torch.einsum("rh,rh->r", hat, v) / h, v.sum(1) / h
    dres = s["dres_out"].double() + rstd[:, None] * (v - level[:, None] - hat * along[:, None])
    return {"dres": dres, "du": dres * _exact_factor(c, s["rng"], *dres.shape),
            "dweight": torch.einsum("rh,rh->h", dy, hat), "dbias": torch.einsum("rh->h", dy)}


def _exact_router(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], s["topk"]
    x = s["logits"].double()
    counted = torch.ones(t, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    logp = torch.log_softmax(x, 1)
    p, lse = logp.exp() * counted[:, None], torch.logsumexp(x, 1) * counted
    if c["op"] == "router":
        # the best one of what is left, K times
        left, picks = x.clone(), []
        for _ in range(k):
            # the first of the largest: argmax of a truth value's first True
            first = (left == left.amax(1, keepdim=True)).int().argmax(1)
            picks.append(first)
            left[torch.arange(t, device="cuda"), first] = -math.inf
        idx = torch.where(counted[:, None], torch.stack(picks, 1), -1)
        hot = torch.stack([(idx == i).sum() for i in range(e)])
    else:
        idx, hot = s["idx"].long(), s["counts"][:e].long()
    n = int(counted.sum())
    f, chosen = hot.double() / (max(n, 1) * k), idx >= 0
    of = torch.gather(logp, 1, idx.clamp(min=0)).masked_fill(~chosen, -math.inf)
    weights = torch.softmax(of, 1) if c["normalize"] else of.exp()
    weights = torch.where(chosen, weights, 0.0)
    if c["op"] == "router":
        loss = BALANCE * e * torch.dot(f, p.sum(0)) / n + Z * torch.dot(lse, lse) / n
        return {"idx": idx.int(), "weights": weights,
                "counts": torch.cat([hot, hot.new_tensor([n])]).int(), "loss": loss.view(1)}
    dloss = s["dloss"].double()
    # gradients with respect to p and to the weights, then through each softmax
    dp = dloss * BALANCE * e / n * f.expand(t, e)
    dw = s["dweights"].double() * chosen
    dl = torch.zeros_like(x)
    onto = torch.zeros(t, e, k, dtype=torch.float64, device="cuda")
    onto.scatter_(1, idx.clamp(min=0)[:, None, :], chosen.double()[:, None, :])
    if c["normalize"]:
        inner = weights * dw - weights * torch.einsum("tk,tk->t", weights, dw)[:, None]
        dl += torch.einsum("tek,tk->te", onto, inner)
    else:
        dp = dp + torch.einsum("tek,tk->te", onto, dw)
    dl += p * dp - p * torch.einsum("te,te->t", p, dp)[:, None]
    return dl + torch.einsum("te,t->te", p, 2 * Z * dloss / n * lse)


def _exact_embedding(s):
    c = s["case"]
    idx, v = s["idx"].long(), c["vocab"]
    inside = ((idx >= 0) & (idx < v)).nonzero()[:, 0]
    if c["op"] == "embedding":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        out[inside] = s["table"][idx[inside]].double().mul_(s["scale"])
        return out
    total = torch.zeros(s["dtable"].shape, dtype=torch.float64, device="cuda")
    total.index_put_((idx[inside],), s["dout"][inside].double(), accumulate=True)
    return total.mul_(s["scale"])
