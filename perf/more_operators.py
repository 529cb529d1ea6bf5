"""The operators in front of, between and beside the expert products of a layer, as they are measured.

Routing to experts with its gradient, the root-mean-square norm with the residual's addition (16-bit and
8-bit results, gradient), the gated activation between the experts' products (16-bit and 8-bit results,
gradient), and low-rank adapters of many requests beside a shared projection.

`own` false: plain torch operations in 32 bits (64 for choices between scores and for codes, where values lie
next to a border), rounded once at the end. `own` true: the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step: 64 sequences choose 8 of 256 experts by sigmoid scores with a balancing bias, from the 4
        # best of 8 groups (latency)
        dict(name="route_decode", op="route", T=64, E=256, K=8, dtype="fp32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, masked=False),
        # the same of a long prefill, an odd number of tokens
        dict(name="route_prefill", op="route", T=16383, E=256, K=8, dtype="fp32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renorm=True, scale=2.5, masked=False),
        # the gradient to the logits in a training step of 4096 tokens, softmax scores of 16-bit logits
        dict(name="route_grad_train", op="route_grad", T=4096, E=128, K=8, dtype="bf16", score="softmax", renorm=True,
             scale=1.0),
        # a decode step's norm: residual added, codes for the experts' 8-bit products and the 16-bit rows for the router
        dict(name="norm_decode", op="norm_int8", T=64, H=7168, dtype="bf16", wide_weight=False, residual=True, y=True),
        # and of a long prefill
        dict(name="norm_prefill", op="norm_int8", T=16384, H=7168, dtype="bf16", wide_weight=False, residual=True, y=True),
        # the norm's gradient in a training step, fp32 weights, with the gradient of the residual stream
        dict(name="norm_grad_train", op="norm_grad", T=4096, H=4096, dtype="bf16", wide_weight=True, residual=True),
        # a decode step's activation between the 8-bit products, 512 routes
        dict(name="act_decode", op="act_int8", T=64, K=8, E=256, total=256, I=2048, dtype="bf16", act="swiglu",
             weights=False),
        # a prefill's under 8-way expert parallelism: one route in eight is here, the router's weight on the input side
        dict(name="act_prefill_ep", op="act_int8", T=16383, K=8, E=32, total=256, I=2048, dtype="bf16", act="swiglu",
             weights=True),
        # its gradient in a training step, with the gradient of the router's weights
        dict(name="act_grad_train", op="act_grad", T=4096, K=8, E=128, total=128, I=2048, dtype="bf16", act="swiglu",
             weights=True),
        # one request's adapter beside a shared expert's gate and up projection, one token (latency)
        dict(name="adapt_one_token", op="adapt", T=1, n=8, r=16, H=7168, N=4096, dtype="bf16", none=0.0),
        # a decode step of 64 requests with 32 adapters, some without one
        dict(name="adapt_decode", op="adapt", T=64, n=32, r=16, H=7168, N=4096, dtype="fp16", none=0.1),
        # a prefill of requests with 16 adapters of rank 64
        dict(name="adapt_prefill", op="adapt", T=16384, n=16, r=64, H=7168, N=4096, dtype="bf16", none=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "norm", "norm_int8", "norm_grad", "act", "act_int8", "act_grad", "adapt"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    T = _log(rng, 1, 16384)
    if op in ("route", "route_grad"):
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * max(2, _log(rng, 8, 512) // G)
        K = rng.randint(1, min(16, E))
        score, renorm = rng.choice(["softmax", "sigmoid"]), K > 1 and rng.random() < 0.7  # (one renormalised weight is 1)
        c = dict(op=op, T=T, E=E, K=K, dtype=dtype, score=score, renorm=renorm, scale=rng.choice([1.0, 2.5]))
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=G, top_groups=rng.randint(max(1, -(-K * G // E)), G),
                     group_top=rng.choice([1, 2]), masked=rng.random() < 0.3)
        return c
    if op in ("norm", "norm_int8", "norm_grad"):
        H = max(1, _log(rng, 64, 16384) // 8 * 8 + rng.choice([0, 0, 0, rng.randint(1, 7)]))
        T = max(1, min(T, 100_000_000 // H))
        c = dict(op=op, T=T, H=H, dtype=dtype, wide_weight=rng.random() < 0.5, residual=rng.random() < 0.6)
        if op == "norm_int8":
            c["y"] = rng.random() < 0.5
        return c
    if op in ("act", "act_int8", "act_grad"):
        total = rng.choice([8, 16, 32, 64, 96, 128, 256])
        E = rng.choice([total, total, max(1, total // 2), max(1, total // 8)]) if T >= 32 else total
        K = rng.randint(1, min(8, total))
        I = max(1, _log(rng, 64, 8192) // 8 * 8 + rng.choice([0, 0, 0, rng.randint(1, 7)]))
        T = max(1, min(T, 60_000_000 // (I * K)))
        return dict(op=op, T=T, K=K, E=E, total=total, I=I, dtype=dtype, act=rng.choice(["swiglu", "swiglu", "relu2"]),
                    weights=rng.random() < 0.5)
    H, N = 16 * _log(rng, 4, 448), _log(rng, 16, 8192)
    r, n = 8 * rng.choice([1, 2, 2, 4, 8, 16]), _log(rng, 1, 64)
    T = max(1, min(T, 90_000_000 // max(H, N), 4_000_000_000 // (n * max(H, N))))
    return dict(op=op, T=T, n=n, r=r, H=H, N=N, dtype=rng.choice(["bf16", "fp16"]), none=rng.choice([0.0, 0.1, 0.5]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape, dtype="fp32", std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(DTYPES[dtype])


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _order(ids, E):
    """The sorted order of the routes, as sort_routes gives it: row_to_route, route_to_row, offsets."""
    key = ids.reshape(-1)
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    keys, perm = torch.sort(key, stable=True)
    offsets = torch.searchsorted(keys, torch.arange(E + 1, device="cuda")).to(torch.int32)
    rows = torch.empty_like(perm)
    rows[perm] = torch.arange(perm.numel(), device="cuda")
    row_to_route = torch.where(keys < E, perm, torch.full_like(perm, -1)).to(torch.int32)
    route_to_row = torch.where(key < E, rows, torch.full_like(rows, -1)).to(torch.int32)
    return row_to_route, route_to_row, offsets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op, s = case, case["op"], dict(case=case)
    T = c["T"]
    if op in ("route", "route_grad"):
        E, K = c["E"], c["K"]
        # some experts more popular than others
        x = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(1, E, generator=g, device="cuda")
        if op == "route":
            if c["masked"]:  # experts that a token must not take, and tokens that must not be routed (padding)
                x = torch.where((_uniform(g, T, E) < 0.1) | (_uniform(g, T, 1) < 0.05), torch.full_like(x, -math.inf), x)
            s["bias"] = _normal(g, E, std=0.05) if c["bias"] else None
        else:
            s["ids"] = (x + 0.1 * torch.randn(T, E, generator=g, device="cuda")).topk(K, dim=1)[1].to(torch.int32)
            s["dweights"] = _normal(g, T, K)
        s["logits"] = x.to(DTYPES[c["dtype"]])
        return s
    if op.startswith("norm"):
        H = c["H"]
        # a few channels carry outliers, as the residual stream's do
        scale = torch.where(_uniform(g, H) < 0.01, 12.0, 1.0)
        s["x"] = (torch.randn(T, H, generator=g, device="cuda") * scale).to(DTYPES[c["dtype"]])
        s["weight"] = (_uniform(g, H) + 0.5).to(torch.float32 if c["wide_weight"] else DTYPES[c["dtype"]])
        s["residual"] = (torch.randn(T, H, generator=g, device="cuda") * scale).to(DTYPES[c["dtype"]]) if c["residual"] else None
        if op == "norm_grad":
            s["dy"] = _normal(g, T, H, dtype=c["dtype"])
        return s
    if op.startswith("act"):
        K, I, R = c["K"], c["I"], T * c["K"]
        logits = torch.randn(T, c["total"], generator=g, device="cuda") + 0.5 * torch.randn(1, c["total"], generator=g, device="cuda")
        top, ids = logits.topk(K, dim=1)
        s["order"] = _order(ids, c["E"])
        s["weights"] = torch.softmax(top, dim=1).contiguous() if c["weights"] else None
        s["h"] = _normal(g, R, I if c["act"] == "relu2" else 2 * I, dtype=c["dtype"])
        if op == "act_int8":
            s["out"], s["scales"] = torch.zeros(R, I, dtype=torch.int8, device="cuda"), torch.zeros(R, device="cuda")
        elif op == "act":
            s["out"] = torch.zeros(R, I, dtype=DTYPES[c["dtype"]], device="cuda")
        else:
            s["da"] = _normal(g, R, I, dtype=c["dtype"])
            s["out"] = torch.zeros_like(s["h"])
        return s
    n, r, H, N = c["n"], c["r"], c["H"], c["N"]
    # requests of unequal length: a few adapters own most tokens
    p = torch.softmax(torch.randn(n, generator=g, device="cuda"), dim=0)
    ids = torch.multinomial(p, T, replacement=True, generator=g)
    ids = torch.where(_uniform(g, T) < c["none"], torch.full_like(ids, -1), ids)
    s["order"] = _order(ids, n)
    off = s["order"][2]
    s["longest"] = max(1, int((off[1:] - off[:-1]).max()))  # most tokens of one adapter, for the padded plain form
    s["x"], s["base"] = _normal(g, T, H, dtype=c["dtype"]), _normal(g, T, N, dtype=c["dtype"])
    s["a"] = _normal(g, n, r, H, dtype=c["dtype"], std=H ** -0.5)
    s["b"] = _normal(g, n, N, r, dtype=c["dtype"], std=r ** -0.5)
    s["scales"] = _uniform(g, n) + 0.5
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_route(s):
    c, x = s["case"], s["logits"].double()  # 64 bits: choices between scores that lie close
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    eligible = x > -math.inf
    if c["score"] == "softmax":
        top = x.amax(dim=1, keepdim=True).clamp(min=torch.finfo(torch.float64).min)
        e = torch.exp(x - top)
        score = e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(eligible, choice, torch.full_like(choice, -math.inf))
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True)[0][:, :, :c["group_top"]]
        has = best[:, :, 0] > -math.inf
        best = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(dim=2)
        best = torch.where(has, best, torch.full_like(best, -math.inf))
        order = best.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        stays = stays[:, :, None].expand(T, G, E // G).reshape(T, E)
        choice = torch.where(stays, choice, torch.full_like(choice, -math.inf))
    value, ids = choice.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :K], ids[:, :K]
    kept = value > -math.inf
    w = torch.where(kept, score.gather(1, ids), torch.zeros_like(value))
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    ids = torch.where(kept, ids, torch.full_like(ids, -1)).to(torch.int32)
    return {"ids": ids, "weights": (w * c["scale"]).float()}


def _plain_route_grad(s):
    c, x = s["case"], s["logits"].float()
    ids, q = s["ids"].long(), s["dweights"] * c["scale"]
    if c["score"] == "softmax":
        score = torch.exp(x - x.amax(dim=1, keepdim=True))
        score = score / score.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    at = score.gather(1, ids)
    if c["renorm"]:
        p = at / at.sum(dim=1, keepdim=True)
        d = p * (q - (p * q).sum(dim=1, keepdim=True))
        d = d if c["score"] == "softmax" else d * (1.0 - at)
        dx = torch.zeros_like(x).scatter_(1, ids, d)
    elif c["score"] == "softmax":
        dx = torch.zeros_like(x).scatter_(1, ids, q)
        dx = score * (dx - (at * q).sum(dim=1, keepdim=True))
    else:
        dx = torch.zeros_like(x).scatter_(1, ids, q * at * (1.0 - at))
    return dx.to(s["logits"].dtype)


def _plain_norm(s):
    c, x = s["case"], s["x"]
    total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    h = total.float()
    r = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    out = {}
    if s["residual"] is not None:
        out["total"] = total
    if c["op"] == "norm" or c["y"]:
        out["y"] = (h * r * s["weight"].float()).to(x.dtype)
    if c["op"] == "norm_int8":
        # r is one positive factor of the row: the codes are those of h w, rounded once to 32 bits
        p = h * s["weight"].float()
        scale = p.abs().amax(dim=1)
        scale = scale / torch.full_like(scale, 127.0)
        # 64 bits: quotients next to a half
        q = p.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]
        out["codes"] = q.round().clamp(-127, 127).to(torch.int8)
        out["scales"] = scale * r[:, 0]
    return out


def _plain_norm_grad(s):
    h, w, dy = s["x"].float(), s["weight"].float(), s["dy"].float()
    r = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    n, g = h * r, dy * w
    dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()  # the gradient that comes down the residual stream
    return {"x": dx.to(s["x"].dtype), "weight": (dy * n).sum(dim=0)}


def _plain_act(s):
    """Rows behind the last route that is here stay 0, as their buffer was."""
    c, h = s["case"], s["h"]
    route, route_to_row, offsets = s["order"]
    R, I = h.shape[0], c["I"]
    here = torch.arange(R, device=h.device) < offsets[-1]
    w = None if s["weights"] is None else s["weights"].reshape(-1)[route.long().clamp(min=0)]
    if c["op"] == "act_int8":
        v = h.double()  # 64 bits: quotients next to a half
        a = torch.square(v.clamp(min=0)) if c["act"] == "relu2" else v[:, :I] / (1.0 + torch.exp(-v[:, :I])) * v[:, I:]
        scale = (a.abs().amax(dim=1) / 127.0).float()
        q = a / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]
        codes = q.round().clamp(-127, 127).to(torch.int8)
        scale = scale if w is None else scale * w
        return {"codes": torch.where(here[:, None], codes, torch.zeros_like(codes)),
                "scales": torch.where(here, scale, torch.zeros_like(scale))}
    v = h.float()
    if c["act"] == "relu2":
        z = v.clamp(min=0)
        a = z * z
    else:
        gate, up = v[:, :I], v[:, I:]
        sig = 1.0 / (1.0 + torch.exp(-gate))
        a = gate * sig * up
    if c["op"] == "act":
        a = a if w is None else a * w[:, None]
        return torch.where(here[:, None], a, torch.zeros_like(a)).to(h.dtype)
    da = s["da"].float()
    d = da if w is None else da * w[:, None]
    if c["act"] == "relu2":
        dh = d * 2.0 * z
    else:
        dh = torch.cat([d * up * (sig + gate * sig * (1.0 - sig)), d * gate * sig], dim=1)
    out = {"h": torch.where(here[:, None], dh, torch.zeros_like(dh)).to(h.dtype)}
    if w is not None:
        dot = (da * a).sum(dim=1)
        row = route_to_row.long()
        out["weights"] = torch.where(row >= 0, dot[row.clamp(min=0)], torch.zeros_like(dot)).view(c["T"], c["K"])
    return out


def _plain_adapt(s):
    c, x = s["case"], s["x"]
    n, T, cap = c["n"], c["T"], s["longest"]
    token, _, offsets = s["order"]
    row = torch.arange(T, device=x.device)
    e = torch.searchsorted(offsets, row, right=True, out_int32=False) - 1
    here = e < n
    e = e.clamp(max=n - 1)
    src = token.long().clamp(min=0)
    at = torch.where(here, e * cap + row - offsets.long()[e], torch.full_like(row, n * cap))
    rows = torch.zeros(n * cap + 1, c["H"], device=x.device)
    rows[at] = x[src].float()
    v = torch.bmm(rows[:-1].view(n, cap, -1), s["a"].float().transpose(1, 2).contiguous())
    d = torch.bmm(v, s["b"].float().transpose(1, 2).contiguous()) * s["scales"][:, None, None]
    d = d.view(n * cap, -1)[at.clamp(max=n * cap - 1)]
    y = s["base"].float()
    y[src[here]] += d[here]
    return y.to(x.dtype)


def _plain(s):
    op = s["case"]["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_grad":
        return _plain_route_grad(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op.startswith("norm"):
        return _plain_norm(s)
    return _plain_act(s) if op.startswith("act") else _plain_adapt(s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import block_scaled_fp4_top_amd as moe
    c = s["case"]
    op = c["op"]
    if op == "route":
        ids, w = moe.route(s["logits"], c["K"], score=c["score"], bias=s["bias"], groups=c["groups"],
                           top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
        return {"ids": ids, "weights": w}
    if op == "route_grad":
        return moe.route_grad(s["dweights"], s["logits"], s["ids"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])
    if op == "norm":
        y, total = moe.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
        return {"y": y} if s["residual"] is None else {"y": y, "total": total}
    if op == "norm_int8":
        y = torch.empty_like(s["x"]) if c["y"] else None
        codes, scales, total = moe.rms_norm_int8(s["x"], s["weight"], EPS, residual=s["residual"], y=y)
        out = {"codes": codes, "scales": scales}
        if c["y"]:
            out["y"] = y
        if s["residual"] is not None:
            out["total"] = total
        return out
    if op == "norm_grad":
        dx, dw = moe.rms_norm_grad(s["dy"], s["x"], s["weight"], EPS, dtotal=s["residual"])
        return {"x": dx, "weight": dw}
    if op == "adapt":
        order = moe.RouteOrder(*s["order"], c["T"], 1, c["n"])
        return moe.adapt(s["base"], s["x"], order, s["a"], s["b"], s["scales"])
    order = moe.RouteOrder(*s["order"], c["T"], c["K"], c["E"])
    if op == "act":
        return moe.activate(s["h"], c["act"], order, s["weights"], out=s["out"])
    if op == "act_int8":
        codes, scales = moe.activate_int8(s["h"], c["act"], order, s["weights"], out=s["out"], scales=s["scales"])
        return {"codes": codes, "scales": scales}
    dh, dw = moe.activate_grad(s["da"], s["h"], c["act"], order, s["weights"], out=s["out"])
    return {"h": dh} if dw is None else {"h": dh, "weights": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    T, b = c["T"], BYTES[c["dtype"]]
    if op == "route":
        return {"bytes": T * c["E"] * b + 8 * T * c["K"] + (4 * c["E"] if c["bias"] else 0), "flops": 4 * T * c["E"]}
    if op == "route_grad":
        dense = c["score"] == "softmax" and not c["renorm"]  # else only the chosen logits count
        read = c["E"] if dense else c["K"]
        return {"bytes": T * (read + c["E"]) * b + 8 * T * c["K"], "flops": 6 * T * (c["E"] if dense else c["K"])}
    if op.startswith("norm"):
        H = c["H"]
        wb = H * (4 if c["wide_weight"] else b)
        if op == "norm_grad":
            return {"bytes": T * H * b * (4 if c["residual"] else 3) + wb + 4 * H, "flops": 9 * T * H}
        n = (3 if c["residual"] else 1) + (1 if op == "norm" or c["y"] else 0)
        return {"bytes": T * H * (n * b + (op == "norm_int8")) + wb + (4 * T if op == "norm_int8" else 0), "flops": 5 * T * H}
    if op.startswith("act"):
        kept = T * c["K"] * c["E"] / c["total"]  # expected share of the routes whose expert is here
        I, two = c["I"], 1 if c["act"] == "relu2" else 2
        w = 8 * kept if c["weights"] else 0
        if op == "act_grad":
            return {"bytes": kept * I * b * (1 + 2 * two) + w + (4 * T * c["K"] if c["weights"] else 0), "flops": 12 * kept * I}
        one = 1 if op == "act_int8" else b
        return {"bytes": kept * (I * (two * b + one) + (4 if op == "act_int8" else 0)) + w, "flops": 6 * kept * I}
    n, r, H, N = c["n"], c["r"], c["H"], c["N"]
    here = T * (1 - c["none"])
    used = min(n, here)  # adapters with tokens, at most
    return {"bytes": here * H * b + 2 * T * N * b + used * r * (H + N) * b, "flops": 2 * here * r * (H + N)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(s):
    c = s["case"]
    x = s["logits"].double()
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    bias = torch.zeros(E, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"].double()
    never = torch.isinf(x) & (x < 0)
    if c["score"] == "sigmoid":
        log_score = -torch.logaddexp(torch.zeros_like(x), -x)
    else:
        log_score = x - torch.logsumexp(x, dim=1, keepdim=True)
    log_score = log_score.masked_fill(never, -math.inf)
    choice = (log_score.exp() + bias).masked_fill(never, -math.inf)
    if G > 1:
        part = choice.reshape(T, G, E // G)
        first = part.max(dim=2)[0]
        total = first.clone()
        if c["group_top"] == 2 and E // G > 1:
            rest = part.clone()
            rest.scatter_(2, part.argmax(dim=2, keepdim=True), -math.inf)
            second = rest.max(dim=2)[0]
            total = total + second.masked_fill(second == -math.inf, 0.0)
        for _ in range(G - c["top_groups"]):  # the worst group goes, of equal ones the last
            low = total.masked_fill(torch.isnan(total), math.inf).min(dim=1, keepdim=True)[0]
            last = torch.where(total == low, torch.arange(G, device="cuda"), -1).max(dim=1, keepdim=True)[0]
            total.scatter_(1, last, math.nan)
        choice = part.masked_fill(torch.isnan(total)[:, :, None], -math.inf).reshape(T, E)
    logs = torch.full((T, K), -math.inf, dtype=torch.float64, device="cuda")
    for k in range(K):
        top = choice.max(dim=1, keepdim=True)[0]
        at = torch.where(choice == top, torch.arange(E, device="cuda"), E).min(dim=1, keepdim=True)[0]
        logs[:, k] = torch.where(top > -math.inf, log_score.gather(1, at), -math.inf)[:, 0]
        choice.scatter_(1, at, -math.inf)
    if c["renorm"]:
        logs = logs - torch.logsumexp(logs, dim=1, keepdim=True).nan_to_num(neginf=0.0)
    return {"ids": None, "weights": logs.exp() * c["scale"]}


def _exact_route_grad(s):
    """Through the Jacobian's products by autograd in 64 bits."""
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    log_score = torch.log_softmax(x, dim=1) if c["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
    at = log_score.gather(1, s["ids"].long())
    w = torch.softmax(at, dim=1) if c["renorm"] else at.exp()
    (w * s["dweights"].double()).sum().mul(c["scale"]).backward()
    return x.grad


def _exact_norm(s):
    c, x, w = s["case"], s["x"], s["weight"].double()
    out = {}
    h = x.double()
    if s["residual"] is not None:
        out["total"] = h + s["residual"].double()
        h = (x + s["residual"]).double()  # the norm reads the stream as it is stored
    size = torch.linalg.vector_norm(h, dim=1, keepdim=True)
    unit = h / torch.sqrt(size * size / c["H"] + EPS)
    if c["op"] == "norm" or c["y"]:
        out["y"] = unit * w
    if c["op"] == "norm_int8":
        out["codes"] = None  # whole numbers
        out["scales"] = torch.linalg.vector_norm(unit * w, ord=math.inf, dim=1) / 127.0
    return out


def _exact_norm_grad(s):
    h, w, dy = (s[k].double() for k in ("x", "weight", "dy"))
    H = h.shape[1]
    rms = torch.sqrt(torch.linalg.vecdot(h, h, dim=1) / H + EPS)[:, None]
    g = dy * w
    dx = g / rms - h * (torch.linalg.vecdot(g, h, dim=1)[:, None] / (H * rms ** 3))
    if s["residual"] is not None:
        dx += s["residual"].double()
    return {"x": dx, "weight": torch.linalg.vecdot(dy, h / rms, dim=0)}


def _exact_act(s):
    c = s["case"]
    route, _, offsets = s["order"]
    kept = int(offsets[-1])
    R, I = c["T"] * c["K"], c["I"]
    at = route[:kept].long()
    h = s["h"][:kept].double().requires_grad_(c["op"] == "act_grad")
    a = torch.relu(h).pow(2) if c["act"] == "relu2" else torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    w = torch.ones(kept, dtype=torch.float64, device="cuda") if s["weights"] is None else s["weights"].double().view(-1)[at]
    if c["op"] == "act":
        out = torch.zeros(R, I, dtype=torch.float64, device="cuda")
        out[:kept] = a * w[:, None]
        return out
    if c["op"] == "act_int8":
        scales = torch.zeros(R, dtype=torch.float64, device="cuda")
        scales[:kept] = torch.linalg.vector_norm(a, ord=math.inf, dim=1) / 127.0 * w
        return {"codes": None, "scales": scales}  # the codes are whole numbers
    da = s["da"][:kept].double()
    a.backward(da * w[:, None])
    dh = torch.zeros(R, h.shape[1], dtype=torch.float64, device="cuda")
    dh[:kept] = h.grad
    if s["weights"] is None:
        return {"h": dh}
    dw = torch.zeros(R, dtype=torch.float64, device="cuda")
    dw[at] = torch.linalg.vecdot(da, a.detach(), dim=1)
    return {"h": dh, "weights": dw.view(c["T"], c["K"])}


def _exact_adapt(s):
    token, _, offsets = s["order"]
    y = s["base"].double()
    bound = offsets.tolist()
    for e in range(s["case"]["n"]):
        at = token[bound[e]:bound[e + 1]].long()
        if at.numel():
            v = s["x"][at].double() @ s["a"][e].double().t().contiguous()
            y[at] += s["scales"][e].double() * (v @ s["b"][e].double().t().contiguous())
    return y


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "route":
        return _exact_route(s)
    if op == "route_grad":
        return _exact_route_grad(s)
    if op == "norm_grad":
        return _exact_norm_grad(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    return _exact_act(s) if op.startswith("act") else _exact_adapt(s)
