"""Cases of the routing, routing-gradient, combine-gradient and adapter operators.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes a case's inputs on the GPU and ``run()`` makes one pass:
the plain torch form of the operator, or (``own``) the calls of
``top_routing_expert_gemm_b200`` that a program makes.  ``exact()`` evaluates
the operator's definition in 64 bits.

Operators
  route        logits [T, E] -> the k experts of each row and their weights
               (sigmoid or softmax scores, selection bias, expert groups)
  route_bwd    the gradient of those weights, of the balance loss and of the
               z-loss with respect to the logits
  combine_bwd  the gradients of the weighted un-permute: of the experts'
               output rows and of the routing weights
  gate_up      h = act(P + s B A x) for rows of many adapters (the experts'
               first projection, P = W x given)
  down         y = base + s B A h (the experts' second projection)
"""
import math

import torch

own = False

SIGMOID, SOFTMAX = "sigmoid", "softmax"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's tokens through a group-limited sigmoid router: latency
        dict(name="route_decode", op="route", T=16, E=256, k=8, score=SIGMOID, bias=True, G=8, Gk=4, gtop=2,
             renorm=True, scale=2.5, dtype="f32", pad=0, mask=False, dead=0),
        # a prefill batch of the same router
        dict(name="route_prefill", op="route", T=8192, E=256, k=8, score=SIGMOID, bias=True, G=8, Gk=4, gtop=2,
             renorm=True, scale=2.5, dtype="f32", pad=0, mask=False, dead=0),
        # a long batch of bf16 logits in padded rows, the last tokens padding, single experts switched off
        dict(name="route_softmax_long", op="route", T=65536, E=128, k=4, score=SOFTMAX, bias=False, G=1, Gk=1,
             gtop=1, renorm=True, scale=1.0, dtype="bf16", pad=8, mask=True, dead=777),
        # a training step's router gradient with both penalties
        dict(name="route_bwd_sigmoid", op="route_bwd", T=8192, E=256, k=8, score=SIGMOID, bias=True, G=8, Gk=4,
             gtop=2, renorm=True, scale=2.5, dtype="f32", pad=0, mask=False, dead=0, balance=True, z=True),
        # an odd expert count and batch, probabilities used as they are
        dict(name="route_bwd_softmax_odd", op="route_bwd", T=4099, E=60, k=6, score=SOFTMAX, bias=False, G=1, Gk=1,
             gtop=1, renorm=False, scale=1.0, dtype="bf16", pad=0, mask=True, dead=3, balance=False, z=True),
        # the combine's gradient at the benchmark's default layer
        dict(name="combine_bwd_2048", op="combine_bwd", T=2048, d=4096, E=8, k=2, dtype="bf16", capacity=0.0),
        # the widest dispatch, with a capacity that drops some slots
        dict(name="combine_bwd_capacity", op="combine_bwd", T=8192, d=2880, E=128, k=4, dtype="bf16", capacity=1.0),
        # the small fp32 layer
        dict(name="combine_bwd_f32", op="combine_bwd", T=256, d=256, E=8, k=2, dtype="f32", capacity=0.0),
        # one token of one request: latency
        dict(name="gate_up_one_token", op="gate_up", T=1, d=4096, f=14336, E=8, k=2, N=16, r=16, dtype="bf16",
             act="swiglu", shared=False, requests=0),
        # a prefill batch of a few requests
        dict(name="gate_up_prefill", op="gate_up", T=2048, d=4096, f=14336, E=8, k=2, N=8, r=16, dtype="bf16",
             act="swiglu", shared=False, requests=12),
        # a decode step, every token of another request: the adapters' weights are the bytes
        dict(name="down_decode", op="down", T=64, d=4096, f=14336, E=8, k=2, N=64, r=16, dtype="bf16",
             act="swiglu", shared=False, requests=0),
        # a prefill batch over many small experts
        dict(name="down_prefill", op="down", T=8192, d=2880, f=2880, E=128, k=4, N=4, r=8, dtype="bf16",
             act="swiglu", shared=False, requests=24),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_route(rng, op):
    G = rng.choice([1, 1, 2, 4, 8])
    E = G * rng.choice([2, 4, 5, 8, 16, 20, 32, 60])
    Gk = rng.randint(1, G)
    k = rng.randint(1, min(16, Gk * (E // G)))
    c = dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=k, score=rng.choice([SIGMOID, SOFTMAX]),
             bias=rng.random() < 0.5, G=G, Gk=Gk, gtop=rng.choice([1, 2]) if E // G > 1 else 1,
             renorm=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
             pad=rng.choice([0, 0, 3, 8]), mask=rng.random() < 0.5)
    c["dead"] = rng.randint(0, c["T"] // 8)
    if op == "route_bwd":
        c["balance"] = rng.random() < 0.5
        c["z"] = rng.random() < 0.5
    return c


def _draw_combine(rng):
    E = rng.choice([4, 8, 32, 128])
    return dict(op="combine_bwd", T=_log_int(rng, 1, 8192), d=8 * _log_int(rng, 1, 512), E=E,
                k=rng.randint(1, min(E, 8)), dtype=rng.choice(["bf16", "bf16", "f32"]),
                capacity=rng.choice([0.0, 0.0, 1.0, 1.25]))


def _draw_adapter(rng, op):
    shared = rng.random() < 0.3
    E = 1 if shared else rng.choice([2, 4, 8, 16, 32, 128])
    T = _log_int(rng, 1, 8192)
    return dict(op=op, T=T, d=8 * _log_int(rng, 8, 512), f=8 * _log_int(rng, 8, 1792), E=E,
                k=1 if shared else rng.randint(1, min(E, 4)), N=_log_int(rng, 1, 64),
                r=8 * rng.choice([1, 2, 2, 3, 4, 8, 16]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                act=rng.choice(["swiglu", "swiglu", "gelu"]), shared=shared,
                requests=rng.choice([0, rng.randint(1, 32)]))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    most_flops = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["route", "route_bwd", "combine_bwd", "gate_up", "down"])
        if op.startswith("route"):
            c = _draw_route(rng, op)
        elif op == "combine_bwd":
            c = _draw_combine(rng)
        else:
            c = _draw_adapter(rng, op)
        w = work(c)
        if w["bytes"] <= most and w["flops"] <= most_flops and _weight_bytes(c) <= 2 << 30:
            return c


def _weight_bytes(c):
    if c["op"] not in ("gate_up", "down"):
        return 0
    n_in, n_out, _ = _widths(c)
    return c["N"] * c["E"] * c["r"] * (n_in + n_out) * (2 if c["dtype"] == "bf16" else 4)


def _widths(c):
    """(columns read by A, columns written by B, columns of the result) of an adapter case."""
    if c["op"] == "down":
        return c["f"], c["d"], c["d"]
    up = 2 * c["f"] if c["act"] == "swiglu" else c["f"]
    return c["d"], up, c["f"]


def work(case):
    c, op = case, case["op"]
    if op in ("route", "route_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        eb = 2 if c["dtype"] == "bf16" else 4
        n = T * E * eb + 8 * T * k + (4 * E if c["bias"] and op == "route" else 0)
        if op == "route":
            return {"bytes": n, "flops": 8 * T * E}
        if not (c["balance"] or c["z"]) and not (c["score"] == SOFTMAX and not c["renorm"]):
            n = T * E * eb + (8 + eb) * T * k  # only the picked logits are read, all gradients are written
        else:
            n += T * E * eb + (4 * E if c["balance"] else 0)
        return {"bytes": n, "flops": 12 * T * E}
    eb = 2 if c["dtype"] == "bf16" else 4
    rows = c["T"] * c["k"]
    if op == "combine_bwd":
        if c["capacity"]:
            rows = min(rows, int(0.93 * rows))  # about what a capacity of the mean load keeps
        return {"bytes": (c["T"] + 2 * rows) * c["d"] * eb + 12 * c["T"] * c["k"], "flops": 3 * rows * c["d"]}
    n_in, n_out, n_res = _widths(c)
    pairs = c["N"] * c["E"]
    touched = pairs * (1.0 - (1.0 - 1.0 / pairs) ** rows) if pairs > 1 else 1.0
    by = rows * (n_in + n_out + n_res) * eb + touched * c["r"] * (n_in + n_out) * eb + 8 * rows
    return {"bytes": int(by), "flops": int(2 * rows * c["r"] * (n_in + n_out))}


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, dtype=torch.float32, std=1.0):
    out = torch.empty(*shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
    return out.to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    if c["op"] in ("route", "route_bwd"):
        st = _prepare_route(c, g)
    elif c["op"] == "combine_bwd":
        st = _prepare_combine(c, g)
    else:
        st = _prepare_adapter(c, g)
    st["case"] = c
    return st


def _prepare_route(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    dt = DTYPES[c["dtype"]]
    wide = _normal(g, T, E + c["pad"], dtype=dt)
    logits = wide[:, :E]
    if c["mask"]:  # experts that a token must not use
        off = torch.rand(T, E, device="cuda", generator=g) < 0.05
        logits.masked_fill_(off, float("-inf"))
    if c["dead"]:  # padding tokens behind the batch: every expert masked with the type's lowest value
        logits[T - c["dead"]:] = torch.finfo(dt).min
    st = dict(logits=logits, bias=_normal(g, E, std=0.1) if c["bias"] else None)
    if c["op"] == "route":
        st["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        st["w"] = torch.empty(T, k, dtype=torch.float32, device="cuda")
    else:
        ids, _ = _route_plain(c, logits, st["bias"])
        st["ids"] = ids
        st["grad_w"] = _normal(g, T, k)
        used = ids[ids >= 0].long()
        st["counts"] = torch.bincount(used, minlength=E).to(torch.int32) if c["balance"] else None
        st["balance"] = 0.01 if c["balance"] else 0.0
        st["z"] = 0.001 if c["z"] else 0.0
        st["grad"] = torch.zeros(T, E + c["pad"], dtype=dt, device="cuda")[:, :E]
    if own:
        import top_routing_expert_gemm_b200 as moe
        st["route"] = moe.make_route_config(
            T, E, k, moe.MOE_SCORE_SIGMOID if c["score"] == SIGMOID else moe.MOE_SCORE_SOFTMAX,
            n_groups=c["G"], topk_groups=c["Gk"], group_top=c["gtop"], renormalise=int(c["renorm"]),
            weight_scale=c["scale"], logits_dtype=moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_F32,
            logits_stride=E + c["pad"])
    return st


def _random_ids(c, g):
    """k distinct experts per token, near the even load of a balanced router."""
    return torch.rand(c["T"], c["E"], device="cuda", generator=g).topk(c["k"], dim=1).indices.to(torch.int32)


def _dispatch(ids, E, capacity):
    """Rows grouped by expert, tokens ascending inside: offsets [E+1], perm and row_of."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    start = torch.cumsum(counts, 0) - counts
    rank = torch.arange(n, device="cuda") - start[flat[order]]
    cap = n if capacity is None else capacity
    kept = counts.clamp(max=cap)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(kept, 0)
    row = torch.where(rank < cap, offsets[flat[order]] + rank, torch.full_like(rank, -1))
    row_of = torch.empty(n, dtype=torch.int64, device="cuda")
    row_of[order] = row
    perm = torch.zeros(n, dtype=torch.int64, device="cuda")
    keep = row_of >= 0
    perm[row_of[keep]] = torch.arange(n, device="cuda")[keep]
    return offsets.to(torch.int32), perm.to(torch.int32), row_of.to(torch.int32)


def _prepare_combine(c, g):
    T, k, d, E = c["T"], c["k"], c["d"], c["E"]
    dt = DTYPES[c["dtype"]]
    cap = None if c["capacity"] == 0 else min(T, math.ceil(T * k / E * c["capacity"]))
    _, _, row_of = _dispatch(_random_ids(c, g), E, cap)
    st = dict(grad_y=_normal(g, T, d, dtype=dt), y_perm=_normal(g, T * k, d, dtype=dt), row_of=row_of,
              w=torch.softmax(_normal(g, T, k), dim=1),
              grad_y_perm=torch.zeros(T * k, d, dtype=dt, device="cuda"),
              grad_w=torch.empty(T, k, dtype=torch.float32, device="cuda"))
    if own:
        import top_routing_expert_gemm_b200 as moe
        st["cfg"] = moe.make_config(T, d, E, k, 8, moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_F32,
                                    moe.MOE_SOFTMAX_TOPK, capacity_factor=c["capacity"])
    return st


def _prepare_adapter(c, g):
    T, k, E, N, r = c["T"], c["k"], c["E"], c["N"], c["r"]
    dt = DTYPES[c["dtype"]]
    n_in, n_out, n_res = _widths(c)
    rows = T * k
    if c["requests"]:  # the tokens of a request follow one another and share its adapter
        cuts = torch.sort(torch.randint(0, T, (c["requests"] - 1,), device="cuda", generator=g)).values
        request = torch.bucketize(torch.arange(T, device="cuda"), cuts, right=True)
    else:              # every token belongs to another request
        request = torch.arange(T, device="cuda")
    # one request in about ten has no adapter
    pick = torch.randint(0, N, (T,), device="cuda", generator=g)
    none = torch.rand(T, device="cuda", generator=g) < 0.1
    token_adapter = torch.where(none, torch.full_like(pick, -1), pick)[request].to(torch.int32)
    st = dict(x=_normal(g, rows, n_in, dtype=dt), base=_normal(g, rows, n_out, dtype=dt),
              token_adapter=token_adapter,
              a=_normal(g, N, E, r, n_in, dtype=dt, std=n_in ** -0.5),
              b=_normal(g, N, E, n_out, r, dtype=dt, std=0.25 * r ** -0.5),
              scale=0.5 + 1.5 * torch.rand(N, device="cuda", generator=g),
              out=torch.empty(rows, n_res, dtype=dt, device="cuda"), offsets=None, perm=None)
    if not c["shared"]:
        st["offsets"], st["perm"], _ = _dispatch(_random_ids(c, g), E, None)
    if own:
        import top_routing_expert_gemm_b200 as moe
        dtype = moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_F32
        act = moe.MOE_ACT_SWIGLU if c["act"] == "swiglu" else moe.MOE_ACT_GELU
        st["cfg"] = moe.make_config(T, c["d"], E, k, c["f"], dtype, moe.MOE_SOFTMAX_TOPK, expert_act=act,
                                    n_shared=int(c["shared"]), d_ff_shared=c["f"] if c["shared"] else 0)
        st["adapters"] = moe.make_adapter_config(N, r, shared=int(c["shared"]))
        st["plan"] = torch.empty(moe.moe_adapter_plan_bytes(st["cfg"], st["adapters"]), dtype=torch.uint8,
                                 device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    c = state["case"]
    if op == "route":
        return _route_plain(c, state["logits"], state["bias"])
    if op == "route_bwd":
        return _route_bwd_plain(c, state)
    if op == "combine_bwd":
        return _combine_bwd_plain(c, state)
    return _adapter_plain(c, state)


def _run_own(st, op):
    import top_routing_expert_gemm_b200 as moe
    if op == "route":
        moe.moe_route_topk(st["route"], st["logits"], st["bias"], st["ids"], st["w"])
        return st["ids"], st["w"]
    if op == "route_bwd":
        moe.moe_route_backward(st["route"], st["logits"], st["ids"], st["grad_w"], st["counts"], st["balance"],
                               st["z"], st["grad"])
        return st["grad"]
    if op == "combine_bwd":
        moe.moe_combine_backward(st["cfg"], st["grad_y"], st["y_perm"], st["row_of"], st["w"], st["grad_y_perm"],
                                 st["grad_w"])
        return st["grad_y_perm"], st["grad_w"]
    moe.moe_adapter_plan(st["cfg"], st["adapters"], st["offsets"], st["perm"], st["token_adapter"], st["plan"])
    apply = moe.moe_adapter_gate_up if op == "gate_up" else moe.moe_adapter_down
    apply(st["cfg"], st["adapters"], st["plan"], st["x"], st["a"], st["b"], st["scale"], st["base"], st["out"])
    return st["out"]


# ------------------------------------------------------------------ plain forms
def _route_plain(c, logits, bias):
    """Selection in 64 bits (scores next to one another decide it), weights in 32."""
    E, G, k = c["E"], c["G"], c["k"]
    avail = logits > torch.finfo(logits.dtype).min
    l = torch.where(avail, logits.double(), torch.full((), float("-inf"), dtype=torch.float64, device="cuda"))
    if c["score"] == SIGMOID:
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        m = l.amax(1, keepdim=True).clamp(min=-1e300)
        e = torch.exp(l - m)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    choice = s if bias is None else s + bias.double()
    choice = torch.where(avail, choice, torch.full_like(choice, float("-inf")))
    if G > 1:
        per = torch.sort(choice.view(-1, G, E // G), dim=2, descending=True).values
        gs = per[:, :, 0]
        if c["gtop"] == 2:  # a group with one expert left counts that one alone
            gs = gs + torch.where(per[:, :, 1] > float("-inf"), per[:, :, 1], torch.zeros_like(gs))
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["Gk"]]
        kept = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, best, True)
        choice = torch.where(kept.repeat_interleave(E // G, dim=1), choice,
                             torch.full_like(choice, float("-inf")))
    val, idx = torch.sort(choice, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    got = val > float("-inf")
    ids = torch.where(got, idx, torch.full_like(idx, -1)).to(torch.int32)
    if c["score"] == SIGMOID:
        w = 1.0 / (1.0 + torch.exp(-l.float()))
    else:
        l32 = l.float()
        e = torch.exp(l32 - l32.amax(1, keepdim=True).clamp(min=-3e38))
        w = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    w = torch.where(got, w.gather(1, idx), torch.zeros((), device="cuda"))
    if c["renorm"]:
        w = w / torch.where(got.any(1, keepdim=True), w.sum(1, keepdim=True), torch.ones((), device="cuda"))
    return ids, w * c["scale"]


def _route_bwd_plain(c, st):
    logits, ids, g = st["logits"], st["ids"], st["grad_w"]
    T, E = c["T"], c["E"]
    avail = logits > torch.finfo(logits.dtype).min
    l = torch.where(avail, logits.float(), torch.full((), float("-inf"), device="cuda"))
    e = torch.exp(l - l.amax(1, keepdim=True).clamp(min=-3e38))
    z = e.sum(1, keepdim=True)
    p = e / z.clamp(min=1e-30)
    got = ids >= 0
    at = ids.clamp(min=0).long()
    g = torch.where(got, g, torch.zeros_like(g)) * c["scale"]
    if c["score"] == SIGMOID:
        s = torch.where(got, torch.sigmoid(l).gather(1, at), torch.zeros_like(g))
        if c["renorm"]:
            q = s / s.sum(1, keepdim=True).clamp(min=1e-30)
            part = q * (1.0 - s) * (g - (q * g).sum(1, keepdim=True))
        else:
            part = g * s * (1.0 - s)
        grad = torch.zeros(T, E, device="cuda").scatter_add_(1, at, torch.where(got, part, torch.zeros_like(part)))
    else:
        s = torch.where(got, p.gather(1, at), torch.zeros_like(g))
        if c["renorm"]:
            q = s / s.sum(1, keepdim=True).clamp(min=1e-30)
            part = q * (g - (q * g).sum(1, keepdim=True))
            grad = torch.zeros(T, E, device="cuda").scatter_add_(1, at, part)
        else:
            grad = torch.zeros(T, E, device="cuda").scatter_add_(1, at, s * g) - p * (s * g).sum(1, keepdim=True)
    if st["balance"]:
        f = st["counts"].float()
        f = f / f.sum().clamp(min=1.0)
        grad = grad + st["balance"] * E / T * p * (f - (p * f).sum(1, keepdim=True))
    if st["z"]:
        lse = torch.where(avail.any(1), torch.log(z[:, 0].clamp(min=1e-30)) + l.amax(1), torch.zeros((), device="cuda"))
        grad = grad + st["z"] * 2.0 / T * lse[:, None] * p
    return torch.where(avail, grad, torch.zeros((), device="cuda")).to(logits.dtype)


def _combine_bwd_plain(c, st):
    T, k = c["T"], c["k"]
    row_of = st["row_of"].long().view(T, k)
    gy = st["grad_y"].float()
    grad_w = torch.zeros(T, k, device="cuda")
    grad_rows = torch.zeros(T * k + 1, c["d"], device="cuda")  # the last row takes the dropped slots
    for s in range(k):
        row = row_of[:, s]
        keep = row >= 0
        prod = gy * st["y_perm"][row.clamp(min=0)].float()
        grad_w[:, s] = torch.where(keep, prod.sum(1), torch.zeros((), device="cuda"))
        grad_rows[torch.where(keep, row, torch.full_like(row, T * k))] = gy * st["w"][:, s:s + 1]
    return grad_rows[:T * k].to(st["grad_y"].dtype), grad_w


def _row_pairs(c, st):
    """Adapter (-1: none) and expert of every row."""
    rows = c["T"] * c["k"]
    if c["shared"]:
        return st["token_adapter"].long(), torch.zeros(rows, dtype=torch.int64, device="cuda")
    adapter = st["token_adapter"][(st["perm"] // c["k"]).long()].long()
    expert = torch.bucketize(torch.arange(rows, device="cuda", dtype=torch.int32), st["offsets"][1:].contiguous(),
                             right=True)
    return adapter, expert


def _adapter_plain(c, st):
    rows = c["T"] * c["k"]
    n_in, n_out, n_res = _widths(c)
    adapter, expert = _row_pairs(c, st)
    out = torch.empty(rows, n_res, dtype=st["base"].dtype, device="cuda")
    step = max(1, (1 << 28) // (c["r"] * max(n_in, n_out)))  # rows whose gathered weights take about 1 GB
    for i in range(0, rows, step):
        a, e = adapter[i:i + step], expert[i:i + step]
        use = (a >= 0).float()[:, None]
        a = a.clamp(min=0)
        u = torch.bmm(st["a"][a, e].float(), st["x"][i:i + step].float()[:, :, None])
        delta = torch.bmm(st["b"][a, e].float(), u)[:, :, 0]
        v = st["base"][i:i + step].float() + use * st["scale"][a][:, None] * delta
        if c["op"] == "gate_up":
            if c["act"] == "swiglu":
                gate, up = v[:, :c["f"]], v[:, c["f"]:]
                v = gate / (1.0 + torch.exp(-gate)) * up
            else:
                v = 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))
        out[i:i + step] = v.to(out.dtype)
    return out


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """``run`` in 64 bits from the definitions: picks one expert after the other,
    gradients from the Jacobians written out, adapters one pair after the other."""
    st = prepare(case, seed)
    c, op = case, case["op"]
    if op == "route":
        return _route_exact(c, st["logits"], st["bias"])
    if op == "route_bwd":
        return _route_bwd_exact(c, st)
    if op == "combine_bwd":
        return _combine_bwd_exact(c, st)
    return _adapter_exact(c, st)


def _log_scores(c, logits):
    """log of every expert's score (-inf: not available)."""
    l = logits.to(torch.float64)
    l = l.masked_fill(~(logits > torch.finfo(logits.dtype).min), -math.inf)
    if c["score"] == SIGMOID:
        return torch.nn.functional.logsigmoid(l).masked_fill(l == -math.inf, -math.inf), l
    lse = torch.logsumexp(l, 1, keepdim=True)
    return torch.where(lse == -math.inf, lse, l - lse), l


def _route_exact(c, logits, bias):
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    ls, l = _log_scores(c, logits)
    choice = torch.exp(ls)
    if bias is not None:
        choice = choice + bias.to(torch.float64)[None]
    choice = choice.masked_fill(l == -math.inf, -math.inf)

    def first_max(v):  # the largest value and the first place that holds it
        m = v.amax(1)
        return m, torch.argmax((v == m[:, None]).to(torch.int8), 1)

    at = torch.arange(T, device="cuda")
    if G > 1:
        rest = choice.reshape(T * G, E // G).clone()
        total = torch.zeros(T * G, dtype=torch.float64, device="cuda")
        for j in range(c["gtop"]):
            m, i = first_max(rest)
            total = total + (m if j == 0 else m.masked_fill(m == -math.inf, 0.0))
            rest[torch.arange(T * G, device="cuda"), i] = -math.inf
        total = total.reshape(T, G)
        open_ = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        for _ in range(c["Gk"]):
            m, i = first_max(total.masked_fill(open_, -math.inf))
            open_[at, i] |= m > -math.inf
        choice = choice.reshape(T, G, E // G).masked_fill(~open_[:, :, None], -math.inf).reshape(T, E)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    lw = torch.full((T, k), -math.inf, dtype=torch.float64, device="cuda")
    choice = choice.clone()
    for j in range(k):
        m, i = first_max(choice)
        ok = m > -math.inf
        ids[:, j] = torch.where(ok, i, torch.full_like(i, -1)).to(torch.int32)
        lw[:, j] = torch.where(ok, ls[at, i], lw[:, j])
        choice[at, i] = -math.inf
    if c["renorm"]:
        lse = torch.logsumexp(lw, 1, keepdim=True)
        lw = torch.where(lse == -math.inf, lse, lw - lse)
    return ids, torch.exp(lw) * c["scale"]


def _route_bwd_exact(c, st):
    T, E, k = c["T"], c["E"], c["k"]
    _, l = _log_scores(c, st["logits"])
    dead = (l == -math.inf).all(1)
    p = torch.softmax(l.masked_fill(dead[:, None], 0.0), 1).masked_fill(dead[:, None], 0.0)
    hot = torch.zeros(T, E, dtype=torch.float64, device="cuda")   # 1 at the picked experts
    up = torch.zeros(T, E, dtype=torch.float64, device="cuda")    # the weights' gradients there
    for j in range(k):
        i = st["ids"][:, j].long()
        ok = (i >= 0).to(torch.float64)
        hot.scatter_add_(1, i.clamp(min=0)[:, None], ok[:, None])
        up.scatter_add_(1, i.clamp(min=0)[:, None], (ok * st["grad_w"][:, j].double())[:, None])
    up = up * c["scale"]
    if c["score"] == SIGMOID:
        s = torch.sigmoid(l)
        ds = s * (1.0 - s)
    else:
        s, ds = p, None
    if c["renorm"]:  # d(s_i / S) = (e_i - s_i / S) / S over the picked ones
        S = (hot * s).sum(1, keepdim=True)
        S = S.masked_fill(S == 0.0, 1.0)
        vs = hot * (up - (up * hot * s).sum(1, keepdim=True) / S) / S
    else:
        vs = hot * up
    if ds is not None:
        grad = vs * ds
    else:
        grad = p * (vs - (p * vs).sum(1, keepdim=True))
    if st["balance"]:
        f = st["counts"].double() / max(1, int(st["counts"].sum()))
        v = (st["balance"] * E / T) * f[None].expand(T, E)
        grad = grad + p * (v - (p * v).sum(1, keepdim=True))
    if st["z"]:
        lse = torch.logsumexp(l.masked_fill(dead[:, None], 0.0), 1, keepdim=True)
        grad = grad + (2.0 * st["z"] / T) * lse * p
    return grad.masked_fill(l == -math.inf, 0.0)


def _combine_bwd_exact(c, st):
    T, k, d = c["T"], c["k"], c["d"]
    row = st["row_of"].long()
    slot = torch.nonzero(row >= 0)[:, 0]
    grad_rows = torch.zeros(T * k, d, dtype=torch.float64, device="cuda")
    grad_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    w = st["w"].double().reshape(-1)
    for part in torch.split(slot, 4096):
        gy = st["grad_y"][part // k].double()
        grad_rows[row[part]] = gy * w[part, None]
        grad_w[part] = torch.einsum("nd,nd->n", gy, st["y_perm"][row[part]].double())
    return grad_rows, grad_w.reshape(T, k)


def _adapter_exact(c, st):
    if c["T"] * c["k"] * _widths(c)[1] > 600_000_000:
        return None
    adapter, expert = _row_pairs(c, st)
    v = st["base"].double()
    pair = torch.where(adapter >= 0, adapter * c["E"] + expert, torch.full_like(adapter, -1))
    for q in torch.unique(pair).tolist():
        if q < 0:
            continue
        a, e = q // c["E"], q % c["E"]
        rows = torch.nonzero(pair == q)[:, 0]
        u = st["x"][rows].double() @ st["a"][a, e].double().T
        v[rows] += st["scale"][a].double() * (u @ st["b"][a, e].double().T)
    if c["op"] == "down":
        return v
    if c["act"] == "swiglu":
        return v[:, :c["f"]] * torch.sigmoid(v[:, :c["f"]]) * v[:, c["f"]:]
    return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
