"""Cases of the mixture-of-experts movement and block-norm operators.

``run`` computes a case in plain torch operations (32-bit arithmetic, one
rounding at the end), or, with ``own`` true, through the library's entry
points.  ``exact`` computes the same from the definitions in 64 bits.

Notation: T tokens, K experts per token, E experts, H hidden size, n = T * K
slots (slot t * K + k), C rows of the sorted buffers.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 0), "e5m2": (torch.float8_e5m2, 57344.0, 1)}
EPS, BRANCH_SCALE, RESIDUAL_SCALE = 1e-6, 0.5, 1.25


# ---------------------------------------------------------------- the cases
def listed():
    def moe(name, op, tokens, topk, experts, hidden, align=16, **more):
        return {"name": name, "op": op, "tokens": tokens, "topk": topk, "experts": experts,
                "hidden": hidden, "align": align, "dtype": "bf16", **more}

    def norm(name, op, rows, hidden, **more):
        return {"name": name, "op": op, "rows": rows, "hidden": hidden, "dtype": "bf16",
                "res": "bf16", "param": "bf16", "gate": "none", "per_gate": 1, "offset": 0.0,
                "fp8": "none", **more}

    return [
        # one decoding step of a small batch: the junction whose output feeds an FP8 product
        norm("norm decode fp8", "norm", 4, 4096, gate="channel", fp8="e4m3"),
        # a training micro-batch with an odd token count, a gate per sequence, gradients kept in fp32 params
        norm("norm train", "norm", 8191, 6144, gate="sequence", per_gate=2048, param="fp32"),
        # odd hidden size, half precision around an fp32 residual stream
        norm("norm backward odd", "norm_bwd", 4099, 777, dtype="fp16", res="fp32", param="fp32",
             offset=1.0),
        # the largest training junction
        norm("norm backward train", "norm_bwd", 8192, 12288, gate="sequence", per_gate=2048),
        # one decoding step: route and gather a handful of tokens, no padding rows
        moe("dispatch decode", "dispatch", 4, 4, 64, 4096, align=1),
        # a training micro-batch into expert order, padded to 16 rows per expert
        moe("dispatch train", "dispatch", 8191, 4, 64, 6144),
        # its gradient: the copies of a token summed
        moe("dispatch backward train", "dispatch_bwd", 8192, 4, 64, 6144),
        # forward of FP8 experts: sorted, cast and transposed in one go
        moe("fp8 dispatch train", "fp8_dispatch", 16384, 4, 64, 6144, fmt="e4m3", weighted=False,
            transpose=True),
        # backward of FP8 experts: the weighted output gradient, cast and transposed
        moe("fp8 dispatch gradient", "fp8_dispatch", 8192, 2, 8, 4096, fmt="e5m2", weighted=True,
            transpose=True),
        # one decoding step: the experts' outputs back to a few tokens
        moe("combine decode", "combine", 4, 4, 64, 4096, align=1),
        # training: weighted sum of eight experts per token
        moe("combine train", "combine", 8192, 8, 128, 4096),
        # its gradient: for the experts' outputs and for the router's weights
        moe("combine backward train", "combine_bwd", 8192, 4, 64, 6144),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _hidden(rng, lo, hi):
    """Half of the draws a multiple of 64, the rest of 8 or any number."""
    h = _log_int(rng, lo, hi)
    step = rng.choice((64, 64, 8, 1))
    h = max(step, h // step * step)
    return h - step if h == 3072 else h


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "dispatch", "dispatch_bwd", "fp8_dispatch", "combine",
                     "combine_bwd"))
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        gate = rng.choice(("none", "channel", "sequence"))
        case = {"op": op, "rows": _log_int(rng, 1, 16384), "hidden": _hidden(rng, 512, 12288),
                "dtype": dtype, "res": rng.choice((dtype, "fp32")),
                "param": rng.choice((dtype, "fp32")), "gate": gate,
                "per_gate": _log_int(rng, 16, 4096) if gate == "sequence" else 1,
                "offset": rng.choice((0.0, 1.0)),
                "fp8": rng.choice(("none", "none", "e4m3", "e5m2")) if op == "norm" else "none"}
        rows = "rows"
    else:
        experts = _log_int(rng, 8, 256)
        case = {"op": op, "tokens": _log_int(rng, 1, 16384), "topk": rng.randint(1, 8),
                "experts": experts, "hidden": _hidden(rng, 512, 12288),
                "align": rng.choice((1, 16, 16, 32, 128)), "dtype": "bf16"}
        if op == "fp8_dispatch":
            case.update(align=rng.choice((1, 16, 16, 32, 128)), fmt=rng.choice(("e4m3", "e5m2")),
                        weighted=rng.random() < 0.5, transpose=rng.random() < 0.75)
        else:
            case["dtype"] = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        rows = "tokens"
    while work(case)["bytes"] > 9e8:
        case[rows] = case[rows] * 3 // 4
    return case


def capacity(c):
    """Rows that hold every token copy whatever the routing: each expert's
    rows are padded to a multiple of `align`, and at most min(E, n) experts
    have any."""
    n = c["tokens"] * c["topk"]
    most = n + min(c["experts"], n) * (c["align"] - 1)
    return -(-most // c["align"]) * c["align"]


def work(c):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    h = c["hidden"]
    if c["op"] in ("norm", "norm_bwd"):
        x, r, t = size[c["dtype"]], size[c["res"]], c["rows"] * h
        if c["op"] == "norm":
            return {"bytes": t * (x + 2 * r + (x if c["fp8"] == "none" else 1)) + 8 * c["rows"],
                    "flops": 10 * t}
        return {"bytes": t * (3 * x + 3 * r) + 8 * c["rows"], "flops": 24 * t}
    b, n = size[c["dtype"]], c["tokens"] * c["topk"]
    one, many, rows = c["tokens"] * h, n * h, capacity(c)
    sort = 8 * n + 4 * rows + 8 * c["experts"]
    if c["op"] == "dispatch":
        return {"bytes": b * (one + rows * h) + sort, "flops": 0}
    if c["op"] == "fp8_dispatch":
        return {"bytes": 2 * one + rows * h * (2 if c["transpose"] else 1) + sort,
                "flops": (2 if c["weighted"] else 1) * many}
    if c["op"] == "combine":
        return {"bytes": b * (one + many) + 8 * n, "flops": 2 * many}
    if c["op"] == "dispatch_bwd":
        return {"bytes": b * (one + many) + 4 * n, "flops": many}
    return {"bytes": b * (one + many + rows * h) + 12 * n, "flops": 3 * many}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    make = _prepare_norm if case["op"] in ("norm", "norm_bwd") else _prepare_moe
    return make(dict(case), g, normal)


def _empty(*shape, dtype):
    return torch.empty(*shape, device="cuda", dtype=dtype)


def _prepare_norm(c, g, normal):
    rows, h = c["rows"], c["hidden"]
    x, r, p = DTYPES[c["dtype"]], DTYPES[c["res"]], DTYPES[c["param"]]
    groups = {"none": 0, "channel": 1}.get(c["gate"], -(-rows // c["per_gate"]))
    c["per_gate"] = rows if c["gate"] == "channel" else c["per_gate"]
    s = {"case": c, "u": normal(rows, h, std=0.7, dtype=x),
         "w_post": normal(h, std=0.2).add_(1 - c["offset"]).to(p),
         "w_pre": normal(h, std=0.2).add_(1 - c["offset"]).to(p),
         "gate": normal(groups, h, std=0.8, dtype=p) if groups else None,
         "rstd_post": _empty(rows, dtype=torch.float32),
         "rstd_pre": _empty(rows, dtype=torch.float32)}
    if c["op"] == "norm":
        s["res"] = normal(rows, h, std=2.0, dtype=r)
        s["res_out"] = torch.empty_like(s["res"])
        s["y"] = _empty(rows, h, dtype=x if c["fp8"] == "none" else torch.uint8)
        if c["fp8"] != "none":  # a delayed scale: from an earlier step's largest output
            s["scale"] = torch.full((1,), FP8[c["fp8"]][1] / 7.0, device="cuda")
            s["amax"], s["scale_inv"] = (torch.zeros(1, device="cuda") for _ in range(2))
        return s
    # what the forward pass has kept, and the two gradients that come back
    s["res_out"] = normal(rows, h, std=2.0, dtype=r)
    s["rstd_post"] = torch.rsqrt(s["u"].float().square().mean(1) + EPS)
    s["rstd_pre"] = torch.rsqrt(s["res_out"].float().square().mean(1) + EPS)
    s["dy"] = normal(rows, h, std=0.05, dtype=x)
    s["dres_out"] = normal(rows, h, std=0.05, dtype=r)
    s["du"], s["dres"] = torch.empty_like(s["u"]), torch.empty_like(s["res_out"])
    for k in ("w_post", "w_pre", "gate"):
        s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
    return s


def _route(c, g, normal):
    """Experts of every token: the most likely K under a router that prefers
    some experts; one token in 50 is padding and goes nowhere (-1)."""
    t, k, e = c["tokens"], c["topk"], c["experts"]
    logits = normal(t, e) + normal(1, e, std=0.8)
    best, idx = torch.topk(logits, k, dim=1)
    away = torch.rand(t, 1, generator=g, device="cuda") < 0.02
    if t < 16:
        away.zero_()
    return torch.where(away, -1, idx).to(torch.int32).contiguous(), torch.softmax(best, 1)


def _prepare_moe(c, g, normal):
    t, k, h, x = c["tokens"], c["topk"], c["hidden"], DTYPES[c["dtype"]]
    idx, weights = _route(c, g, normal)
    rows, op = capacity(c), c["op"]
    s = {"case": c, "idx": idx, "weights": weights}
    if op in ("dispatch", "fp8_dispatch"):
        s["x"] = normal(t, h, dtype=x)
        if op == "dispatch":
            s["out"] = _empty(rows, h, dtype=x)
            return s
        s["out"] = _empty(rows, h, dtype=torch.uint8)
        s["out_t"] = _empty(h, rows, dtype=torch.uint8) if c["transpose"] else None
        s["scale"] = torch.full((1,), FP8[c["fmt"]][1] / 5.5, device="cuda")
        s["amax"], s["scale_inv"] = (torch.zeros(1, device="cuda") for _ in range(2))
        return s
    s.update(zip(("row_of", "src", "offsets", "counts"), _plain_sort(idx, c["experts"], c["align"],
                                                                     rows)))
    if op == "combine_bwd":
        s["ys"], s["dout"] = normal(rows, h, dtype=x), normal(t, h, std=0.05, dtype=x)
        s["dys"], s["dweights"] = torch.empty_like(s["ys"]), torch.empty_like(weights)
    else:
        s["ys"] = normal(rows, h, std=1.0 if op == "combine" else 0.05, dtype=x)
        s["out"] = _empty(t, h, dtype=x)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_sort(idx, experts, align, rows):
    """Stable order by expert.  row_of[t, k]: the sorted row of the slot (-1:
    dropped); src[row]: its slot (-1: padding)."""
    flat = idx.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    key = key[order]
    count = torch.zeros(experts + 1, dtype=torch.long, device=idx.device)
    count.scatter_add_(0, key, torch.ones_like(key))
    padded = (count[:experts] + align - 1) // align * align
    offsets = torch.zeros(experts + 2, dtype=torch.long, device=idx.device)
    offsets[1:experts + 1] = padded.cumsum(0)
    first = count.cumsum(0) - count
    row = offsets[key] + torch.arange(n, device=idx.device) - first[key]
    row = torch.where((key < experts) & (row < rows), row, -1)
    row_of = torch.empty_like(flat).scatter_(0, order, row)
    src = torch.full((rows + 1,), -1, dtype=torch.long, device=idx.device)
    src.scatter_(0, torch.where(row >= 0, row, rows), order)
    return (row_of.view(idx.shape).int(), src[:rows].int(), offsets[:experts + 1].int(),
            count[:experts].int())


def _plain_fp8(v, scale, fmt):
    dtype, top, _ = FP8[fmt]
    return (v * scale).clamp(-top, top).to(dtype)


def _plain_moe(s):
    c = s["case"]
    op, k = c["op"], c["topk"]
    if op in ("dispatch", "fp8_dispatch"):
        row_of, src, offsets, counts = _plain_sort(s["idx"], c["experts"], c["align"], capacity(c))
        slot = src.long()
        rows = torch.where((slot >= 0)[:, None], s["x"][slot.clamp(min=0) // k].float(), 0.0)
        plan = {"row_of": row_of, "src": src, "offsets": offsets, "counts": counts}
        if op == "dispatch":
            return {"out": rows.to(s["x"].dtype), **plan}
        if c["weighted"]:
            rows = rows * s["weights"].reshape(-1)[slot.clamp(min=0)][:, None]
        q = _plain_fp8(rows, s["scale"], c["fmt"])
        out = {"out": q, "amax": torch.maximum(s["amax"], rows.abs().max()),
               "scale_inv": 1.0 / s["scale"], **plan}
        if c["transpose"]:
            out["out_t"] = q.t().contiguous()
        return out
    row, kept = s["row_of"].long().clamp(min=0), (s["row_of"] >= 0)[:, :, None]
    if op == "combine_bwd":
        slot = s["src"].long()
        at = slot.clamp(min=0)
        dout = s["dout"].float()
        each = dout[at // k] * s["weights"].reshape(-1)[at][:, None]
        dys = torch.where((slot >= 0)[:, None], each, 0.0).to(s["ys"].dtype)
        dots = (s["ys"][row].float() * dout[:, None]).sum(2)
        return {"dys": dys, "dweights": torch.where(kept[:, :, 0], dots, 0.0)}
    parts = torch.where(kept, s["ys"][row].float(), 0.0)
    if op == "combine":
        parts = parts * s["weights"][:, :, None]
    return parts.sum(1).to(s["ys"].dtype)


def _gate_rows(s):
    """The gate's row of every row, or 1 without a gate."""
    if s["gate"] is None:
        return 1.0
    rows = torch.arange(s["u"].shape[0], device="cuda") // s["case"]["per_gate"]
    return s["gate"].float()[rows]


def _plain_norm(s):
    c = s["case"]
    u, gate = s["u"].float(), _gate_rows(s)
    w_post, w_pre = s["w_post"].float() + c["offset"], s["w_pre"].float() + c["offset"]
    if c["op"] == "norm":
        rstd_post = torch.rsqrt((u * u).mean(1) + EPS)
        res = RESIDUAL_SCALE * s["res"].float() + BRANCH_SCALE * gate * (u * rstd_post[:, None]
                                                                          * w_post)
        rstd_pre = torch.rsqrt((res * res).mean(1) + EPS)
        y = res * rstd_pre[:, None] * w_pre
        out = {"res_out": res.to(s["res"].dtype), "rstd_post": rstd_post, "rstd_pre": rstd_pre}
        if c["fp8"] == "none":
            return {"y": y.to(s["u"].dtype), **out}
        return {"y": _plain_fp8(y, s["scale"], c["fp8"]),
                "amax": torch.maximum(s["amax"], y.abs().max()), "scale_inv": 1.0 / s["scale"],
                **out}
    dy, hat = s["dy"].float(), s["res_out"].float() * s["rstd_pre"][:, None]
    back = dy * w_pre
    total = s["dres_out"].float() + s["rstd_pre"][:, None] * (
        back - hat * (back * hat).mean(1, keepdim=True))
    hat_u = u * s["rstd_post"][:, None]
    dz = BRANCH_SCALE * gate * total
    back = dz * w_post
    du = s["rstd_post"][:, None] * (back - hat_u * (back * hat_u).mean(1, keepdim=True))
    out = {"du": du.to(s["u"].dtype), "dres": (RESIDUAL_SCALE * total).to(s["dres"].dtype),
           "dw_pre": (dy * hat).sum(0).to(s["w_pre"].dtype),
           "dw_post": (dz * hat_u).sum(0).to(s["w_post"].dtype)}
    if s["gate"] is not None:
        each = BRANCH_SCALE * total * hat_u * w_post
        rows = torch.arange(each.shape[0], device="cuda") // c["per_gate"]
        dgate = torch.zeros(s["gate"].shape, device="cuda").index_add_(0, rows, each)
        out["dgate"] = dgate.to(s["gate"].dtype)
    return out


# ---------------------------------------------------------------- the library
def _own_moe(s):
    import cast_transpose_gb300 as ct
    c = s["case"]
    op = c["op"]
    plan = s.get("plan")
    if plan is None:  # a program keeps one for its batch shape
        have = {b: s[b] for b in ("row_of", "src", "offsets", "counts") if b in s}
        plan = s["plan"] = ct.MoePlan(c["tokens"], c["topk"], c["experts"], align=c["align"],
                                      **have)
    if op in ("dispatch", "fp8_dispatch"):
        ct.moe_sort(s["idx"], plan)
        of_plan = {"row_of": plan.row_of, "src": plan.src, "offsets": plan.offsets,
                   "counts": plan.counts}
        if op == "dispatch":
            ct.moe_dispatch(s["x"], plan, s["out"])
            return {"out": s["out"], **of_plan}
        dtype, _, fmt = FP8[c["fmt"]]
        ct.fp8_moe_dispatch(s["x"], plan, s["scale"], s["amax"], s["scale_inv"], s["out"],
                            s["out_t"], fmt, weights=s["weights"] if c["weighted"] else None)
        out = {"out": s["out"].view(dtype), "amax": s["amax"], "scale_inv": s["scale_inv"],
               **of_plan}
        if c["transpose"]:
            out["out_t"] = s["out_t"].view(dtype)
        return out
    if op == "combine":
        ct.moe_combine(s["ys"], plan, s["weights"], s["out"])
        return s["out"]
    if op == "dispatch_bwd":
        ct.moe_dispatch_backward(s["ys"], plan, s["out"])
        return s["out"]
    ct.moe_combine_backward(s["dout"], s["ys"], plan, s["weights"], s["dys"], s["dweights"])
    return {"dys": s["dys"], "dweights": s["dweights"]}


def _own_norm(s):
    import cast_transpose_gb300 as ct
    c = s["case"]
    same = {"w_post": s["w_post"], "w_pre": s["w_pre"], "gate": s["gate"],
            "rows_per_gate": c["per_gate"], "weight_offset": c["offset"],
            "branch_scale": BRANCH_SCALE, "residual_scale": RESIDUAL_SCALE}
    if c["op"] == "norm":
        out = {"res_out": s["res_out"], "rstd_post": s["rstd_post"], "rstd_pre": s["rstd_pre"]}
        if c["fp8"] == "none":
            ct.block_norm(s["u"], s["res"], y=s["y"], eps=EPS, **same, **out)
            return {"y": s["y"], **out}
        dtype, _, fmt = FP8[c["fp8"]]
        ct.block_norm(s["u"], s["res"], y=s["y"], eps=EPS, scale=s["scale"], amax=s["amax"],
                      scale_inv=s["scale_inv"], fmt=fmt, **same, **out)
        return {"y": s["y"].view(dtype), "amax": s["amax"], "scale_inv": s["scale_inv"], **out}
    if "workspace" not in s:
        size = ct.block_norm_backward_workspace_size(c["rows"], c["hidden"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = {k: s[k] for k in ("du", "dres", "dw_post", "dw_pre", "dgate")}
    ct.block_norm_backward(s["dy"], s["dres_out"], s["u"], s["res_out"], s["rstd_post"],
                           s["rstd_pre"], workspace=s["workspace"], **same, **out)
    return {k: v for k, v in out.items() if v is not None}


def run(state):
    norm = state["case"]["op"] in ("norm", "norm_bwd")
    if own:
        return _own_norm(state) if norm else _own_moe(state)
    return _plain_norm(state) if norm else _plain_moe(state)


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] in ("norm", "norm_bwd") else _exact_moe(s)


def _count_before(idx, experts):
    """For every slot the number of earlier slots of its expert, by counting."""
    flat = idx.reshape(-1).long()
    hot = flat[:, None] == torch.arange(experts, device=flat.device)
    upto = torch.empty(hot.shape, dtype=torch.int32, device=flat.device)
    torch.cumsum(hot, 0, dtype=torch.int32, out=upto)
    return flat, (upto * hot).sum(1) - 1, upto[-1].long()


def _exact_plan(s):
    c = s["case"]
    rows = capacity(c)
    flat, rank, counts = _count_before(s["idx"], c["experts"])
    groups = -(-counts // c["align"]) * c["align"]
    offsets = torch.cat([groups.new_zeros(1), torch.cumsum(groups, 0)])
    row = torch.full_like(flat, -1)
    goes = (flat >= 0) & (flat < c["experts"])
    row[goes] = offsets[flat[goes]] + rank[goes]
    src = torch.full((rows,), -1, dtype=torch.long, device="cuda")
    src[row[goes]] = goes.nonzero()[:, 0]
    return row, src, offsets, counts


def _exact_moe(s):
    c = s["case"]
    op, k, h = c["op"], c["topk"], c["hidden"]
    row, src, offsets, counts = _exact_plan(s)
    slots = (row >= 0).nonzero()[:, 0]
    at = row[slots]
    if op in ("dispatch", "fp8_dispatch"):
        plan = {"row_of": row.view(-1, k).int(), "src": src.int(), "offsets": offsets.int(),
                "counts": counts.int()}
        out = torch.zeros(capacity(c), h, dtype=torch.float64, device="cuda")
        out[at] = s["x"].double()[slots // k]
        if op == "dispatch":
            return {"out": out, **plan}
        if c["weighted"]:
            out[at] *= s["weights"].double().reshape(-1, 1)[slots]
        dtype, top, _ = FP8[c["fmt"]]
        amax = out.abs().max().reshape(1)
        out.mul_(s["scale"].double()).clamp_(-top, top)
        q = out.to(dtype).double()
        both = {"out": q, "amax": amax, "scale_inv": 1 / s["scale"].double(), **plan}
        if c["transpose"]:
            both["out_t"] = q.t().contiguous()
        return both
    if op in ("combine", "dispatch_bwd"):
        total = torch.zeros(c["tokens"], h, dtype=torch.float64, device="cuda")
        each = s["ys"][at].double()
        if op == "combine":
            each *= s["weights"].double().reshape(-1, 1)[slots]
        return total.index_add_(0, slots // k, each)
    dout = s["dout"].double()
    dys = torch.zeros(s["ys"].shape, dtype=torch.float64, device="cuda")
    dys[at] = dout[slots // k] * s["weights"].double().reshape(-1, 1)[slots]
    dw = torch.zeros(c["tokens"] * k, dtype=torch.float64, device="cuda")
    dw[slots] = torch.einsum("nh,nh->n", s["ys"][at].double(), dout[slots // k])
    return {"dys": dys, "dweights": dw.view(-1, k)}


def _exact_norm(s):
    c = s["case"]
    rows, h = s["u"].shape
    u = s["u"].double()
    a_post, a_pre = (s[w].double() + c["offset"] for w in ("w_post", "w_pre"))
    group = torch.arange(rows, device="cuda") // c["per_gate"]
    a_gate = BRANCH_SCALE * (s["gate"].double()[group] if s["gate"] is not None
                             else torch.ones(1, 1, dtype=torch.float64, device="cuda"))
    if c["op"] == "norm":
        post = 1 / torch.sqrt(torch.linalg.vector_norm(u, dim=1).square() / h + EPS)
        res = torch.addcmul(RESIDUAL_SCALE * s["res"].double(), a_gate * a_post,
                            u * post[:, None])
        pre = 1 / torch.sqrt(torch.linalg.vector_norm(res, dim=1).square() / h + EPS)
        y = res * (pre[:, None] * a_pre)
        out = {"res_out": res, "rstd_post": post, "rstd_pre": pre}
        if c["fp8"] == "none":
            return {"y": y, **out}
        dtype, top, _ = FP8[c["fp8"]]
        q = (y * s["scale"].double()).clamp(-top, top).to(dtype).double()
        return {"y": q, "amax": y.abs().max().reshape(1), "scale_inv": 1 / s["scale"].double(),
                **out}
    # gradients of the two norms from their Jacobian: J v = rstd v - x (x . v) rstd^3 / H
    def norm_gradient(x, rstd, v):
        along = torch.einsum("rh,rh->r", x, v) * rstd.pow(3) / h
        return v * rstd[:, None] - x * along[:, None]

    res, dy = s["res_out"].double(), s["dy"].double()
    pre, post = s["rstd_pre"].double(), s["rstd_post"].double()
    down = s["dres_out"].double() + norm_gradient(res, pre, dy * a_pre)
    out = {"du": norm_gradient(u, post, down * a_gate * a_post), "dres": RESIDUAL_SCALE * down,
           "dw_pre": torch.einsum("rh,rh,r->h", dy, res, pre),
           "dw_post": torch.einsum("rh,rh->h", down * a_gate, u * post[:, None])}
    if s["gate"] is not None:
        each = down * u * post[:, None] * (BRANCH_SCALE * a_post)
        out["dgate"] = torch.stack([each[i * c["per_gate"]:(i + 1) * c["per_gate"]].sum(0)
                                    for i in range(s["gate"].shape[0])])
    return out
