"""Cases of the operators around the expert layer, for timing and comparing them.

Three groups of operators, one pass each:

  route      router logits [T, E] to each token's K experts and weights, and the
             gradient of the logits from that of the weights;
  permute    token rows [T, H] copied to the rows of their experts (sorted as the
             compact dispatch sorts them), and the gradient of the token rows;
  unpermute  expert rows summed back per token with the routing weights, and the
             gradients of the rows and of the weights;
  adapters   out[t] = x[t] W^T + scale_l (x[t] A_l^T) B_l^T with l the adapter of
             token t (-1: none), or the second term added to a given projection.

`own` False computes the operators from elementary torch operations in 32 bits;
`own` True calls this repository's kernels.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _device():
    return torch.device("cuda", torch.cuda.current_device())


def listed():
    return [
        # one decode step of 128 tokens: the router's smallest call
        dict(name="route_decode", op="route", T=128, E=384, K=6, dtype="bf16", renorm=True,
             grad=False, pad=0.1),
        # a training micro-batch with float32 router logits, forward and backward
        dict(name="route_train", op="route", T=8192, E=384, K=6, dtype="f32", renorm=True,
             grad=True, pad=0.0),
        # a large batch whose weights are the softmax over all experts
        dict(name="route_large", op="route", T=65536, E=384, K=6, dtype="bf16", renorm=False,
             grad=True, pad=0.02),
        # decode on one of eight expert-parallel ranks: few rows, latency
        dict(name="permute_decode", op="permute", T=128, H=7168, K=6, E=384, local=48,
             dtype="bf16", grad=False, pad=0.1),
        # a training micro-batch with every expert here, forward and backward
        dict(name="permute_train", op="permute", T=8192, H=7168, K=6, E=384, local=384,
             dtype="bf16", grad=True, pad=0.0),
        # decode in half precision, the rows of 96 of 384 experts summed back
        dict(name="unpermute_decode", op="unpermute", T=128, H=5120, K=6, E=384, local=96,
             dtype="f16", grad=False, pad=0.1),
        # float32 rows of one of four ranks, an odd token count, padded slots
        dict(name="unpermute_share", op="unpermute", T=4095, H=5120, K=6, E=384, local=96,
             dtype="f32", grad=True, pad=0.1),
        # the training micro-batch on the way back: out, rows' and weights' gradients
        dict(name="unpermute_train", op="unpermute", T=8192, H=7168, K=6, E=384, local=384,
             dtype="bf16", grad=True, pad=0.0),
        # one sequence decoding with its adapter: the weight's bytes count
        dict(name="adapters_one", op="adapters", T=1, H=5120, N=4608, L=8, rank=16,
             dtype="bf16", weight=True, mixed=True, none=0.0),
        # 128 sequences decoding together, 64 adapters among them
        dict(name="adapters_decode", op="adapters", T=128, H=7168, N=7168, L=64, rank=32,
             dtype="bf16", weight=True, mixed=True, none=0.1),
        # prompts of many requests packed one after the other
        dict(name="adapters_prompts", op="adapters", T=8191, H=7168, N=7168, L=16, rank=64,
             dtype="bf16", weight=True, mixed=False, none=0.1),
        # adapters alone, added to a projection computed elsewhere
        dict(name="adapters_added", op="adapters", T=4097, H=2304, N=5120, L=96, rank=8,
             dtype="f16", weight=False, mixed=False, none=0.1),
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "permute", "unpermute", "adapters", "adapters"])
    if op == "route":
        return dict(op=op, T=_between(rng, 1, 65536), E=_between(rng, 8, 512), K=rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "f16", "f32"]), renorm=rng.random() < 0.5,
                    grad=rng.random() < 0.6, pad=rng.choice([0.0, 0.02, 0.1]))
    if op in ("permute", "unpermute"):
        dtype = rng.choice(["bf16", "f16", "f32"])
        E = _between(rng, 8, 384)
        return dict(op=op, T=_between(rng, 1, 4096), H=_between(rng, 128, 7168, 128),
                    K=rng.randint(1, 8), E=E, local=max(1, E // rng.choice([1, 1, 2, 4, 8])),
                    dtype=dtype, grad=rng.random() < 0.6, pad=rng.choice([0.0, 0.05, 0.1]))
    return dict(op=op, T=_between(rng, 1, 8191), H=_between(rng, 512, 7168, 128),
                N=_between(rng, 128, 7168, 8), L=_between(rng, 1, 64),
                rank=rng.choice([8, 16, 24, 32, 64]), dtype=rng.choice(["bf16", "bf16", "f16"]),
                weight=rng.random() < 0.75, mixed=rng.random() < 0.4,
                none=rng.choice([0.0, 0.1, 0.5]))


# ---- inputs --------------------------------------------------------------------------


def _normal(gen, shape, dtype, std=1.0):
    v = torch.empty(shape, dtype=torch.float32, device=gen.device).normal_(0.0, std, generator=gen)
    return v.to(dtype)


def _uniform(gen, shape, lo=0.0, hi=1.0):
    return torch.rand(shape, generator=gen, device=gen.device) * (hi - lo) + lo


def _tables(case, gen):
    """Routes of T tokens and the compact dispatch's tables of them: each expert's routes
    together, in the order of their slots; -1 for slots that go nowhere here."""
    T, K, E, local = case["T"], case["K"], case["E"], case["local"]
    ids = torch.argsort(_uniform(gen, (T, E)), dim=1)[:, :min(K, E)]
    if K > E:
        ids = torch.cat([ids, ids[:, :K - E]], 1)
    ids = torch.where(_uniform(gen, (T, K)) < case["pad"], -1, ids)
    key = torch.where((ids >= 0) & (ids < local), ids, local).reshape(-1)
    order = torch.argsort(key, stable=True)
    n = int((key < local).sum())
    row_route = torch.full((T * K,), -1, dtype=torch.int32, device=gen.device)
    route_row = torch.full((T * K,), -1, dtype=torch.int32, device=gen.device)
    row_route[:n] = order[:n].to(torch.int32)
    route_row[order[:n]] = torch.arange(n, dtype=torch.int32, device=gen.device)
    w = torch.softmax(_normal(gen, (T, K), torch.float32), dim=1)
    return row_route, route_row, n, w.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    dev, T = gen.device, case["T"]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        l = _normal(gen, (T, E), torch.float32)
        # padded tokens arrive with every logit at -inf
        l = torch.where(_uniform(gen, (T, 1)) < case["pad"], float("-inf"), l)
        s["logits"] = l.to(dt)
        s["dw"] = _normal(gen, (T, K), torch.float32)
        s["ids"] = torch.empty((T, K), dtype=torch.int32, device=dev)
        s["w"] = torch.empty((T, K), dtype=torch.float32, device=dev)
        s["dlogits"] = torch.empty((T, E), dtype=dt, device=dev)
    elif case["op"] in ("permute", "unpermute"):
        H, K = case["H"], case["K"]
        s["row_route"], s["route_row"], s["used"], s["w"] = _tables(case, gen)
        s["x"] = _normal(gen, (T, H), dt)           # token rows, or their gradient
        s["rows"] = _normal(gen, (T * K, H), dt)    # expert rows, or their gradient
        # rows that hold no route stay as they are here: zero
        s["to_rows"] = torch.zeros((T * K, H), dtype=dt, device=dev)
        s["to_x"] = torch.empty((T, H), dtype=dt, device=dev)
        s["to_w"] = torch.empty((T, K), dtype=torch.float32, device=dev)
    else:
        H, N, L, r = case["H"], case["N"], case["L"], case["rank"]
        s["x"] = _normal(gen, (T, H), dt)
        s["weight"] = _normal(gen, (N, H), dt, H ** -0.5) if case["weight"] else None
        s["a"] = _normal(gen, (L, r, H), dt, H ** -0.5)
        s["b"] = _normal(gen, (L, N, r), dt, 0.5 * r ** -0.5)
        s["scale"] = _uniform(gen, (L,), 0.5, 2.0)
        if case["mixed"]:
            ids = torch.randint(0, L, (T,), generator=gen, device=dev)
            ids = torch.where(_uniform(gen, (T,)) < case["none"], -1, ids)
        else:
            # requests of different lengths one after the other, about 300 tokens each
            q = max(1, T // 300)
            cuts = torch.randint(0, T, (q,), generator=gen, device=dev)
            of = torch.randint(0, L, (q + 1,), generator=gen, device=dev)
            of = torch.where(_uniform(gen, (q + 1,)) < case["none"], -1, of)
            at = torch.arange(T, device=dev)
            ids = of[(at[:, None] >= cuts[None, :]).sum(1)]
        s["ids"] = ids.to(torch.int32)
        s["out"] = torch.empty((T, N), dtype=dt, device=dev)
        s["base"] = None if case["weight"] else _normal(gen, (T, N), dt)
    return s


# ---- one pass --------------------------------------------------------------------------


def _plan(s):
    """The shape (and workspace) that a program keeps for its calls."""
    import dispatch_grouped_gemm_amd as moe
    c = s["case"]
    if c["op"] == "route":
        plan = moe, moe.MoeShape(T=c["T"], H=128, I=128, K=c["K"], E_total=c["E"],
                                 E_local=min(c["E"], 512)), None
    elif c["op"] in ("permute", "unpermute"):
        plan = moe, moe.MoeShape(T=c["T"], H=c["H"], I=128, K=c["K"], E_total=c["E"],
                                 E_local=c["local"]), None
    else:
        shape = moe.AdapterShape(T=c["T"], H=c["H"], N=c["N"], L=c["L"], rank=c["rank"])
        plan = moe, shape, moe.alloc_adapter_workspace(shape, s["x"].device)
    s["plan"] = plan
    return plan


def _run_own(s):
    c = s["case"]
    moe, shape, ws = s.get("plan") or _plan(s)
    if c["op"] == "route":
        moe.moe_route(shape, s["logits"], s["ids"], s["w"], renormalize=c["renorm"])
        if not c["grad"]:
            return [s["ids"], s["w"]]
        moe.moe_route_backward(shape, s["logits"], s["ids"], s["w"], s["dw"], s["dlogits"],
                               renormalize=c["renorm"])
        return [s["ids"], s["w"], s["dlogits"]]
    if c["op"] == "permute":
        moe.moe_permute(shape, s["x"], s["route_row"], s["to_rows"])
        if not c["grad"]:
            return [s["to_rows"]]
        moe.moe_permute_backward(shape, s["rows"], s["route_row"], s["to_x"])
        return [s["to_rows"], s["to_x"]]
    if c["op"] == "unpermute":
        moe.moe_unpermute(shape, s["rows"], s["w"], s["route_row"], s["to_x"])
        if not c["grad"]:
            return [s["to_x"]]
        moe.moe_unpermute_backward(shape, s["x"], s["rows"], s["w"], s["route_row"], s["to_rows"],
                                   s["to_w"])
        return [s["to_x"], s["to_rows"], s["to_w"]]
    moe.moe_adapter_project(shape, s["x"], s["weight"], s["ids"], s["a"], s["b"], s["scale"],
                            s["out"], ws, base=s["base"])
    return [s["out"]]


def _exp_to_max(l, m):
    """exp(l - m) with 1 where l is m, infinite or not."""
    return torch.exp(torch.where(l == m, torch.zeros_like(l), l - m))


def _route(s):
    c = s["case"]
    l = s["logits"].float()
    there = l > float("-inf")                       # false for NaN too
    l = torch.where(there, l, float("-inf"))
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    K = c["K"]
    if K > c["E"]:
        val = torch.nn.functional.pad(val, (0, K - c["E"]), value=float("-inf"))
        idx = torch.nn.functional.pad(idx, (0, K - c["E"]))
    val, idx = val[:, :K], idx[:, :K]
    kept = val > float("-inf")
    m = val[:, :1]
    e = torch.where(kept, _exp_to_max(val, m), 0.0)
    every = torch.where(there, _exp_to_max(l, m), 0.0)
    total = (e if c["renorm"] else every).sum(1, keepdim=True)
    w = torch.where(kept, e / total, 0.0)
    ids = torch.where(kept, idx, -1).to(torch.int32)
    if not c["grad"]:
        return [ids, w]
    g = torch.where(kept, s["dw"], 0.0)
    dot = (w * g).sum(1, keepdim=True)
    at = torch.where(kept, idx, 0)
    if c["renorm"]:
        d = torch.zeros_like(l).scatter_add_(1, at, torch.where(kept, w * (g - dot), 0.0))
    else:
        dense = torch.zeros_like(l).scatter_add_(1, at, g)
        d = torch.where(there, every / total * (dense - dot), 0.0)
    return [ids, w, d.to(s["logits"].dtype)]


def _sum_rows(rows, w, route_row, T, K):
    """sum over k of w[t, k] rows[route_row[t, k]], slots of -1 left out."""
    rr = route_row.reshape(T, K).long()
    v = rows[rr.clamp(min=0)].float()
    v = torch.where((rr >= 0)[:, :, None], v if w is None else v * w[:, :, None], 0.0)
    return v.sum(1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _route(s)
    T = c["T"]
    if c["op"] in ("permute", "unpermute"):
        K, n, dt = c["K"], s["used"], s["x"].dtype
        route = s["row_route"][:n].long()
        token = torch.div(route, K, rounding_mode="floor")
        if c["op"] == "permute":
            s["to_rows"][:n] = s["x"][token]
            if not c["grad"]:
                return [s["to_rows"]]
            return [s["to_rows"], _sum_rows(s["rows"], None, s["route_row"], T, K).to(dt)]
        out = _sum_rows(s["rows"], s["w"], s["route_row"], T, K).to(dt)
        if not c["grad"]:
            return [out]
        g = s["x"].float()
        s["to_rows"][:n] = (s["w"].reshape(-1)[route][:, None] * g[token]).to(dt)
        rr = s["route_row"].reshape(T, K).long()
        dw = (g[:, None, :] * s["rows"][rr.clamp(min=0)].float()).sum(2)
        return [out, s["to_rows"], torch.where(rr >= 0, dw, 0.0)]
    L, r = c["L"], c["rank"]
    x = s["x"].float()
    ids = s["ids"].long()
    # every adapter's product for every token, the other adapters' parts put to zero
    v = (x @ s["a"].float().reshape(L * r, -1).t()).reshape(T, L, r)
    mine = ids[:, None] == torch.arange(L, device=ids.device)[None, :]
    v = torch.where(mine[:, :, None], v * s["scale"][None, :, None], 0.0).reshape(T, L * r)
    d = v @ s["b"].float().permute(0, 2, 1).reshape(L * r, -1)
    base = s["base"].float() if s["base"] is not None else x @ s["weight"].float().t()
    return [(base + d).to(s["x"].dtype)]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    T, b = case["T"], BYTES[case["dtype"]]
    if case["op"] == "route":
        E, K = case["E"], case["K"]
        byt = T * E * b + 8 * T * K                       # logits; ids and weights
        if case["grad"]:
            # the weights' gradient in, the logits' out
            byt += 4 * T * K + T * E * b
        return dict(bytes=byt, flops=4 * T * E * (2 if case["grad"] else 1))
    if case["op"] in ("permute", "unpermute"):
        H, K = case["H"], case["K"]
        kept = T * K * (1 - case["pad"]) * case["local"] / case["E"]
        rows, tok = kept * H * b, T * H * b
        if case["op"] == "permute":
            byt = rows + tok + 4 * T * K
            return dict(bytes=byt * (2 if case["grad"] else 1) - (4 * T * K if case["grad"] else 0),
                        flops=kept * H if case["grad"] else 0)
        byt = rows + tok + 8 * T * K
        if case["grad"]:
            byt += tok + rows + 4 * T * K
        return dict(bytes=byt, flops=kept * H * (5 if case["grad"] else 2))
    H, N, L, r = case["H"], case["N"], case["L"], case["rank"]
    with_one = T * (1 - case["none"])
    groups = with_one if case["mixed"] else min(with_one, max(1, T // 300) + 1)
    used = L * (1 - (1 - 1 / L) ** groups)                # different adapters, on average
    byt = T * H * b + T * N * b + used * r * (H + N) * b + 4 * T + 4 * L
    byt += N * H * b if case["weight"] else T * N * b
    return dict(bytes=byt, flops=(2 * T * N * H if case["weight"] else 0)
                + 2 * with_one * r * (H + N))


# ---- the definition in 64 bits ---------------------------------------------------------


def _exact_route(s):
    c = s["case"]
    T, E, K = c["T"], c["E"], c["K"]
    l = s["logits"].double()
    # one whole number per logit that orders them, equal ones by the lower index
    uniq, rank = torch.unique(l, return_inverse=True)
    key = rank.reshape(T, E) * E + (E - 1 - torch.arange(E, device=l.device))[None, :]
    key = torch.where(torch.isneginf(l) | torch.isnan(l), -1, key)
    top = torch.topk(key, min(K, E), dim=1).values
    if K > E:
        top = torch.cat([top, top.new_full((T, K - E), -1)], 1)
    ids = torch.where(top >= 0, E - 1 - top % E, -1)
    p = torch.exp(l - l.max(1, keepdim=True).values)
    p = torch.where(torch.isneginf(l), 0.0, p)
    chosen = torch.zeros((T, E + 1), dtype=torch.bool, device=l.device)
    chosen.scatter_(1, torch.where(ids >= 0, ids, E), True)
    chosen = chosen[:, :E]
    if c["renorm"]:
        p = torch.where(chosen, p, 0.0)
    p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    w = torch.where(ids >= 0, torch.gather(p, 1, ids.clamp(min=0)), 0.0)
    if not c["grad"]:
        return [ids.to(torch.int32), w]
    g = torch.zeros((T, E + 1), dtype=torch.float64, device=l.device)
    g.scatter_(1, torch.where(ids >= 0, ids, E), s["dw"].double())
    g = torch.where(chosen, g[:, :E], 0.0)
    return [ids.to(torch.int32), w, p * (g - (p * g).sum(1, keepdim=True))]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    T = case["T"]
    if case["op"] in ("permute", "unpermute"):
        H, K = case["H"], case["K"]
        rr = s["route_row"].long()
        slot = torch.nonzero(rr >= 0)[:, 0]
        row, tok = rr[slot], torch.div(slot, K, rounding_mode="floor")
        w = s["w"].double().reshape(-1)
        per = torch.zeros((T, H), dtype=torch.float64, device=rr.device)
        y = s["rows"][row].double()
        if case["op"] == "permute":
            to = s["to_rows"].double()
            to[row] = s["x"].double()[tok]
            return [to, per.index_add_(0, tok, y)] if case["grad"] else [to]
        out = per.index_add_(0, tok, y * w[slot][:, None])
        if not case["grad"]:
            return [out]
        g = s["x"].double()[tok]
        to = s["to_rows"].double()
        to[row] = g * w[slot][:, None]
        dw = torch.zeros(T * K, dtype=torch.float64, device=rr.device)
        dw[slot] = (g * y).sum(1)
        return [out, to, dw.reshape(T, K)]
    x = s["x"].double()
    out = s["base"].double() if s["base"] is not None else x @ s["weight"].double().t()
    for l in range(case["L"]):
        at = torch.nonzero(s["ids"] == l)[:, 0]
        v = x[at] @ s["a"][l].double().t()
        out[at] += float(s["scale"][l]) * (v @ s["b"][l].double().t())
    return [out]
