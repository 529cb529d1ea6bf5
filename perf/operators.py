"""The operators around the experts of a Mixture-of-Experts layer, as they are measured.

Routes sorted by expert, token rows dispatched to the experts' rows and combined back (with the router's
weights, and the gradients of both), activations quantized to 8-bit integers, and the dense and the grouped
8-bit integer products.

`own` false: plain torch operations in 32 bits (64 where a value lies next to a rounding border), rounded once
at the end. `own` true: the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step's routes: 64 sequences, 256 experts on this GPU (latency)
        dict(name="sort_decode", op="sort", T=64, K=8, E=256, total=256, ids="int32"),
        # a prefill's routes under 8-way expert parallelism: 32 of 256 experts are here, the other routes are
        # dropped; ids as torch.topk gives them, an odd number of tokens
        dict(name="sort_prefill_ep", op="sort", T=16383, K=8, E=32, total=256, ids="int64"),
        # token rows copied to their experts' rows before the experts' products of a long prefill
        dict(name="dispatch_prefill", op="dispatch", T=16384, H=7168, K=8, E=256, total=256, dtype="bf16", weights=False),
        # its gradient in fp16 training with the router weight on the input side; ragged count, a quarter of the
        # experts elsewhere
        dict(name="dispatch_grad_ep", op="dispatch_grad", T=2047, H=2048, K=6, E=48, total=64, dtype="fp16", weights=True),
        # one decode step's combine: 64 tokens, wide rows
        dict(name="combine_decode", op="combine", T=64, H=7168, K=8, E=256, total=256, dtype="bf16", weights=True),
        # the combine's gradient in a training step of 4096 tokens
        dict(name="combine_grad_train", op="combine_grad", T=4096, H=4096, K=8, E=128, total=128, dtype="bf16", weights=True),
        # activations of a decode batch before the 8-bit product
        dict(name="quantize_decode", op="quantize", T=256, H=2048, dtype="fp16"),
        # and of a long prefill
        dict(name="quantize_prefill", op="quantize", T=16384, H=7168, dtype="bf16"),
        # one token through a dense projection (a shared expert's down projection): weight streaming
        dict(name="matmul_one_token", op="matmul", T=1, N=7168, H=2048, dtype="bf16", bias=False),
        # a prefill through a dense projection (a shared expert's gate and up projection)
        dict(name="matmul_prefill", op="matmul", T=16384, N=4096, H=7168, dtype="bf16", bias=True),
        # the experts' gate and up projections of one decode step: most of 256 experts get a few rows
        dict(name="grouped_decode", op="grouped", T=64, N=4096, H=7168, K=8, E=256, total=256, dtype="bf16", gather=True),
        # and of a prefill, in fp16
        dict(name="grouped_prefill", op="grouped", T=4096, N=4096, H=4096, K=8, E=128, total=128, dtype="fp16", gather=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch_grad", "combine", "combine_grad", "quantize", "matmul", "grouped"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    total = rng.choice([8, 16, 32, 64, 96, 128, 256])
    E = rng.choice([total, total, max(1, total // 2), max(1, total // 8)])
    K = rng.randint(1, min(8, total))
    T = _log(rng, 1, 16384)
    if op == "sort":
        return dict(op=op, T=T, K=K, E=E, total=total, ids=rng.choice(["int32", "int64"]))
    if op == "quantize":
        return dict(op=op, T=T, H=_log(rng, 64, 14336) // rng.choice([1, 8]) + 1, dtype=dtype)
    if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        H = max(1, _log(rng, 64, 7168) // 8 * 8 + rng.choice([0, 0, 0, rng.randint(1, 7)]))
        T = max(1, min(T, 400_000_000 // (H * K)))
        return dict(op=op, T=T, H=H, K=K, E=E, total=total, dtype=dtype, weights=rng.random() < 0.7)
    N, H = _log(rng, 16, 8192), 16 * _log(rng, 4, 448)
    if op == "matmul":
        return dict(op=op, T=T, N=N, H=H, dtype=dtype, bias=rng.random() < 0.5)
    E = min(E, max(1, 2_000_000_000 // (N * H)))
    total = min(total, 8 * E)
    K = min(K, total)
    T = max(1, min(T, 400_000_000 // (max(N, H) * K), int(5e14 // (2 * N * H * K))))
    return dict(op=op, T=T, N=N, H=H, K=K, E=E, total=total, dtype=dtype, gather=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape, dtype="fp32"):
    return torch.randn(*shape, generator=g, device="cuda").to(DTYPES[dtype])


def _codes(g, *shape):
    """8-bit codes as a quantizer leaves them: a normal's values, the largest of some hundred at 127."""
    out = torch.empty(*shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1, shape[-1])
    step = max(1, (1 << 28) // shape[-1])
    for i in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - i)
        v = torch.randn(n, shape[-1], generator=g, device="cuda", dtype=torch.float16)
        flat[i:i + n] = v.mul_(38).round_().clamp_(-127, 127).to(torch.int8)
    return out


def _scales(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda") * 0.02 + 0.005


def _routes(g, c):
    """Router picks: K different experts of `total` for each token, some experts more popular than others, and
    softmax weights. Experts 0..E-1 are on this GPU; the others' ids are E and more."""
    logits = torch.randn(c["T"], c["total"], generator=g, device="cuda")
    logits = logits + 0.5 * torch.randn(1, c["total"], generator=g, device="cuda")
    top, ids = logits.topk(c["K"], dim=1)
    return ids, torch.softmax(top, dim=1)


def _order(ids, E):
    """The sorted order of the routes (what a program that dispatches has in hand)."""
    key = ids.reshape(-1)
    key = torch.where(key < E, key, torch.full_like(key, E))
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
    if op == "sort":
        s["ids"] = _routes(g, c)[0].to(torch.int32 if c["ids"] == "int32" else torch.int64).contiguous()
        return s
    if op == "quantize":
        # a few channels carry outliers, as the inputs of projections do
        x = torch.randn(c["T"], c["H"], generator=g, device="cuda")
        x = x * torch.where(torch.rand(c["H"], generator=g, device="cuda") < 0.01, 12.0, 1.0)
        s["x"] = x.to(DTYPES[c["dtype"]])
        return s
    if op == "matmul":
        s["a"], s["sa"] = _codes(g, c["T"], c["H"]), _scales(g, c["T"])
        s["b"], s["sb"] = _codes(g, c["N"], c["H"]), _scales(g, c["N"])
        s["bias"] = _normal(g, c["N"]) if c["bias"] else None
        return s
    ids, w = _routes(g, c)
    s["order"] = _order(ids, c["E"])
    s["weights"] = w.contiguous() if c.get("weights") else None
    R = c["T"] * c["K"]
    if op == "grouped":
        s["a"] = _codes(g, c["T"] if c["gather"] else R, c["H"])
        s["sa"] = _scales(g, c["T"] if c["gather"] else R)
        s["b"], s["sb"] = _codes(g, c["E"], c["N"], c["H"]), _scales(g, c["E"], c["N"])
        off = s["order"][2]
        s["longest"] = max(1, int((off[1:] - off[:-1]).max()))  # most rows of one expert, for the padded plain form
        s["out"] = torch.zeros(R, c["N"], dtype=DTYPES[c["dtype"]], device="cuda")
    elif op in ("dispatch", "combine_grad"):
        s["tokens"] = _normal(g, c["T"], c["H"], dtype=c["dtype"])
        if op == "combine_grad":
            s["rows"] = _normal(g, R, c["H"], dtype=c["dtype"])
        s["out"] = torch.zeros(R, c["H"], dtype=DTYPES[c["dtype"]], device="cuda")
    else:
        s["rows"] = _normal(g, R, c["H"], dtype=c["dtype"])
        s["tokens"] = _normal(g, c["T"], c["H"], dtype=c["dtype"]) if op == "dispatch_grad" else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_sort(ids, E):
    key = ids.reshape(-1)
    here = (key >= 0) & (key < E)
    key = torch.where(here, key, torch.full_like(key, E))
    keys, perm = torch.sort(key, stable=True)
    offsets = torch.searchsorted(keys, torch.arange(E + 1, device=ids.device, dtype=keys.dtype)).to(torch.int32)
    rows = torch.empty_like(perm)
    rows[perm] = torch.arange(perm.numel(), device=ids.device)
    row_to_route = torch.where(keys < E, perm, torch.full_like(perm, -1)).to(torch.int32)
    route_to_row = torch.where(here, rows, torch.full_like(rows, -1)).to(torch.int32)
    return {"row_to_route": row_to_route, "route_to_row": route_to_row, "offsets": offsets}


def _plain_scatter(tokens, order, w, K):
    """Rows of the experts from the tokens' rows: out[row(t, k)] = w[t, k] tokens[t], 0 behind the last row."""
    route = order[0].long()
    kept = (route >= 0)[:, None]
    route = route.clamp(min=0)
    rows = tokens[route // K].float()
    if w is not None:
        rows = rows * w.reshape(-1)[route][:, None]
    return torch.where(kept, rows, torch.zeros_like(rows)).to(tokens.dtype)


def _plain_gather(rows, order, T, K):
    """The rows of each token's routes in 32 bits, [T, K, H], 0 for a dropped route."""
    row = order[1].long().view(T, K)
    got = rows[row.clamp(min=0)].float()
    return torch.where((row >= 0)[:, :, None], got, torch.zeros_like(got))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "sort":
        return _plain_sort(s["ids"], c["E"])
    if op == "quantize":
        x = s["x"].float()
        scale = x.abs().amax(dim=1)
        scale = scale / torch.full_like(scale, 127.0)
        q = x.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]
        # 64 bits: quotients next to a half. The codes are integers, returned and compared as such
        return {"codes": q.round().clamp(-127, 127).to(torch.int8), "scales": scale}
    if op == "matmul":
        y = (s["a"].float() @ s["b"].float().t()) * s["sa"][:, None] * s["sb"][None, :]
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(DTYPES[c["dtype"]])
    if op == "grouped":
        route, _, offsets = s["order"]
        E, N, cap, R = c["E"], c["N"], s["longest"], route.numel()
        row = torch.arange(R, device=route.device)
        e = torch.searchsorted(offsets, row, right=True, out_int32=False) - 1
        kept = e < E
        e = e.clamp(max=E - 1)
        src = route.long().clamp(min=0) // c["K"] if c["gather"] else row
        at = torch.where(kept, e * cap + row - offsets.long()[e], torch.full_like(row, E * cap))
        a = torch.zeros(E * cap + 1, c["H"], device=route.device)
        a[at] = s["a"][src].float()
        y = torch.bmm(s["b"].float(), a[:-1].view(E, cap, -1).transpose(1, 2).contiguous())  # [E, N, cap]
        y = y.transpose(1, 2).reshape(E * cap, N)[at.clamp(max=E * cap - 1)]
        y = y * s["sa"][src][:, None] * s["sb"][e]
        return torch.where(kept[:, None], y, torch.zeros_like(y)).to(DTYPES[c["dtype"]])
    if op == "dispatch":
        return _plain_scatter(s["tokens"], s["order"], s["weights"], c["K"])
    if op == "combine_grad":
        drows = _plain_scatter(s["tokens"], s["order"], s["weights"], c["K"])
        if s["weights"] is None:
            return {"rows": drows}
        got = _plain_gather(s["rows"], s["order"], c["T"], c["K"])
        return {"rows": drows, "weights": (got * s["tokens"].float()[:, None, :]).sum(dim=2)}
    got = _plain_gather(s["rows"], s["order"], c["T"], c["K"])
    w = s["weights"]
    y = (got if w is None else got * w[:, :, None]).sum(dim=1).to(s["rows"].dtype)
    if op == "combine":
        return y
    if w is None:
        return {"tokens": y}
    return {"tokens": y, "weights": (got * s["tokens"].float()[:, None, :]).sum(dim=2)}


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import block_scaled_fp4_top_amd as moe
    c = s["case"]
    op = c["op"]
    if op == "sort":
        o = moe.sort_routes(s["ids"], c["E"])
        return {"row_to_route": o.row_to_route, "route_to_row": o.route_to_row, "offsets": o.offsets}
    if op == "quantize":
        codes, scales = moe.quantize_int8(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "matmul":
        return moe.int8_matmul(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], out_dtype=DTYPES[c["dtype"]])
    order = moe.RouteOrder(*s["order"], c["T"], c["K"], c["E"])
    if op == "grouped":
        return moe.int8_grouped_matmul(s["a"], s["sa"], s["b"], s["sb"], order, gather=c["gather"], out=s["out"])
    w = s["weights"]
    if op == "dispatch":
        return moe.dispatch(s["tokens"], order, w, out=s["out"])
    if op == "combine":
        return moe.combine(s["rows"], order, w)
    if op == "combine_grad":
        drows, dw = moe.combine_grad(s["tokens"], order, s["rows"] if w is not None else None, w, out=s["out"])
        return {"rows": drows} if dw is None else {"rows": drows, "weights": dw}
    dx, dw = moe.dispatch_grad(s["rows"], order, s["tokens"] if w is not None else None, w)
    return {"tokens": dx} if dw is None else {"tokens": dx, "weights": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, op = case, case["op"]
    T = c["T"]
    if op == "sort":
        R = T * c["K"]
        return {"bytes": R * (4 if c["ids"] == "int32" else 8) + 8 * R + 4 * (c["E"] + 1), "flops": 0}
    if op == "quantize":
        return {"bytes": T * c["H"] * (BYTES[c["dtype"]] + 1) + 4 * T, "flops": 2 * T * c["H"]}
    if op == "matmul":
        N, H = c["N"], c["H"]
        return {"bytes": (T + N) * (H + 4) + (4 * N if c["bias"] else 0) + T * N * BYTES[c["dtype"]], "flops": 2 * T * N * H}
    R = T * c["K"]
    kept = R * c["E"] / c["total"]  # expected share of the routes whose expert is here
    if op == "grouped":
        N, H = c["N"], c["H"]
        used = c["E"] * (1 - (1 - c["K"] / c["total"]) ** T)  # expected number of experts with rows
        rows = (T if c["gather"] else kept) * (H + 4)
        return {"bytes": rows + used * N * (H + 4) + kept * N * BYTES[c["dtype"]], "flops": 2 * kept * N * H}
    H, b = c["H"], BYTES[c["dtype"]]
    small = 4 * R + (4 * R if c["weights"] else 0)
    n = {"dispatch": T + kept, "combine": T + kept,
         "dispatch_grad": T + kept + (T if c["weights"] else 0),
         "combine_grad": T + kept + (kept if c["weights"] else 0)}[op]
    dw = 4 * R if c["weights"] and op.endswith("grad") else 0
    return {"bytes": n * H * b + small + dw, "flops": 2 * kept * H * (2 if dw else 1)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c, op = case, case["op"]
    if op == "sort":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "quantize":
        top = torch.linalg.vector_norm(s["x"].double(), ord=math.inf, dim=1)
        return {"codes": None, "scales": top / torch.full_like(top, 127.0)}  # the codes are whole numbers
    if op == "matmul":
        out = torch.empty(c["T"], c["N"], dtype=torch.float64, device="cuda")
        bt = s["b"].double().t().contiguous() * s["sb"].double()
        for i in range(0, c["T"], 4096):
            out[i:i + 4096] = (s["a"][i:i + 4096].double() @ bt) * s["sa"][i:i + 4096].double()[:, None]
        return out if s["bias"] is None else out + s["bias"].double()
    row_to_route, route_to_row, offsets = (v.long() for v in s["order"])
    K, T = c["K"], c["T"]
    R = T * K
    if op == "grouped":
        out = torch.zeros(R, c["N"], dtype=torch.float64, device="cuda")
        bound = offsets.tolist()
        for e in range(c["E"]):
            lo, hi = bound[e], bound[e + 1]
            if lo < hi:
                at = row_to_route[lo:hi] // K if c["gather"] else torch.arange(lo, hi, device="cuda")
                left = s["a"][at].double() * s["sa"][at].double()[:, None]
                out[lo:hi] = left @ (s["b"][e].double() * s["sb"][e].double()[:, None]).t().contiguous()
        return out
    kept = int(offsets[-1])
    route = row_to_route[:kept]
    token = torch.div(route, K, rounding_mode="floor")
    w = None if s["weights"] is None else s["weights"].double().reshape(-1)[route]

    def rows_of_tokens():
        out = torch.zeros(R, c["H"], dtype=torch.float64, device="cuda")
        got = s["tokens"].double()[token]
        out[:kept] = got if w is None else got * w[:, None]
        return out

    def dots():
        out = torch.zeros(R, dtype=torch.float64, device="cuda")
        out[route] = torch.linalg.vecdot(s["rows"][:kept].double(), s["tokens"].double()[token], dim=1)
        return out.view(T, K)

    def sums():
        got = s["rows"][:kept].double()
        out = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, token, got if w is None else got * w[:, None])

    if op == "dispatch":
        return rows_of_tokens()
    if op == "combine":
        return sums()
    name = "rows" if op == "combine_grad" else "tokens"
    first = rows_of_tokens() if op == "combine_grad" else sums()
    return {name: first} if w is None else {name: first, "weights": dots()}
