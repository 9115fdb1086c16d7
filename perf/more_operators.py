"""Cases of the dense feed-forward block beside the experts, for timing and comparing them.

Three groups of operators, one pass each:

  ffn     the block that every token takes next to its experts (a shared expert, or a
          dense layer): h = silu(min(g, limit)) clamp(u, limit) with g | u = x W13^T, and
          out = h W2^T (+ the experts' output); for training also its gradients, from the
          pre-activations g | u that the forward pass keeps in the elements' type;
  keep8   the same training step with both activations that it keeps in 8 bits: g | u as
          MX FP8 from the forward pass, x as the MX FP8 rows that the experts take;
  norm    the residual joint around a block: res = skip x + scale sigmoid(gate_t) post(y),
          normed = pre(res), both RMS norms with weights, in one pass; and its gradients.

`own` False computes the operators from elementary torch operations in 32 bits;
`own` True calls this repository's kernels.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


def _device():
    return torch.device("cuda", torch.cuda.current_device())


def listed():
    return [
        # one sequence decoding: the weights' bytes count
        dict(name="ffn_one", op="ffn", T=1, H=5120, I=2304, dtype="bf16", base=False,
             limit=10.0, grad=False),
        # 128 sequences decoding together, added to what the experts gave
        dict(name="ffn_decode", op="ffn", T=128, H=7168, I=2048, dtype="bf16", base=True,
             limit=10.0, grad=False),
        # one short prompt in half precision, an odd length, a narrow block
        dict(name="ffn_short", op="ffn", T=509, H=5120, I=1536, dtype="f16", base=True,
             limit=10.0, grad=False),
        # prompts of many requests packed one after the other
        dict(name="ffn_prompts", op="ffn", T=8191, H=7168, I=2048, dtype="bf16", base=True,
             limit=10.0, grad=False),
        # a training micro-batch, forward and backward
        dict(name="ffn_train", op="ffn", T=4096, H=5120, I=2304, dtype="bf16", base=False,
             limit=10.0, grad=True),
        # a small one with an odd length and limits that some values reach
        dict(name="ffn_train_short", op="ffn", T=1021, H=2304, I=1408, dtype="f16", base=False,
             limit=4.0, grad=True),
        # a large micro-batch that keeps 8 bits of its activations
        dict(name="keep8_train", op="keep8", T=8192, H=7168, I=2048, dtype="bf16", base=False,
             limit=10.0, grad=True),
        # the small one in half precision, 8 bits kept
        dict(name="keep8_short", op="keep8", T=1021, H=2304, I=1408, dtype="f16", base=False,
             limit=10.0, grad=True),
        # a decode step's joint after the block and before the next: latency
        dict(name="norm_decode", op="norm", T=128, H=7168, dtype="bf16", y=True, post=True,
             gate=True, skip=1.0, scale=1.0, grad=False),
        # a training micro-batch's joint, the forward pass
        dict(name="norm_train", op="norm", T=8192, H=7168, dtype="bf16", y=True, post=True,
             gate=True, skip=1.0, scale=0.5, grad=False),
        # its gradients: rows, gates and both weights
        dict(name="norm_train_back", op="norm", T=8192, H=7168, dtype="bf16", y=True, post=True,
             gate=True, skip=1.0, scale=0.5, grad=True),
        # float32 rows before a block (no joint), an odd count, the gradients
        dict(name="norm_pre_back", op="norm", T=4095, H=5120, dtype="f32", y=False, post=False,
             gate=False, skip=1.0, scale=1.0, grad=True),
    ]


def _between(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn", "keep8", "norm", "norm"])
    if op == "norm":
        y = rng.random() < 0.75
        return dict(op=op, T=_between(rng, 1, 8192), H=_between(rng, 128, 7168, 32),
                    dtype=rng.choice(["bf16", "f16", "f32"]), y=y,
                    post=y and rng.random() < 0.6, gate=y and rng.random() < 0.6,
                    skip=rng.choice([1.0, 1.0, 2.0]), scale=rng.choice([1.0, 0.5, 0.22]),
                    grad=rng.random() < 0.5)
    grad = op == "keep8" or rng.random() < 0.4
    return dict(op=op, T=_between(rng, 16 if op == "keep8" else 1, 8191),
                H=_between(rng, 256, 7168, 32), I=_between(rng, 128, 2304, 32),
                dtype=rng.choice(["bf16", "bf16", "f16"]), base=not grad and rng.random() < 0.5,
                limit=rng.choice([10.0, 10.0, 4.0]), grad=grad)


# ---- inputs --------------------------------------------------------------------------


def _normal(gen, shape, dtype, std=1.0):
    v = torch.empty(shape, dtype=torch.float32, device=gen.device).normal_(0.0, std, generator=gen)
    return v.to(dtype)


def _mx_rows(v):
    """Rows [T, N] as MX FP8: e4m3 codes and one power of two for 32 values."""
    b = v.float().reshape(v.shape[0], -1, 32)
    e = torch.frexp(b.abs().amax(2, keepdim=True)).exponent - 9
    codes = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.reshape(v.shape).view(torch.uint8), (e[:, :, 0] + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    dt, dev = DTYPES[case["dtype"]], gen.device
    T, H = case["T"], case["H"]
    s = dict(case=case)
    if case["op"] == "norm":
        s["w_pre"] = 1.0 + _normal(gen, (H,), torch.float32, 0.1)
        s["w_pre"] = s["w_pre"].to(dt)
        # the residual stream has a few channels much larger than the rest
        wide = torch.where(torch.rand(H, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        x = _normal(gen, (T, H), torch.float32) * wide
        s["y"] = _normal(gen, (T, H), dt, 0.7) if case["y"] else None
        s["w_post"] = (1.0 + _normal(gen, (H,), torch.float32, 0.1)).to(dt) if case["post"] else None
        s["gate"] = _normal(gen, (T,), torch.float32) if case["gate"] else None
        if not case["grad"]:
            s["x"] = x.to(dt)
            s["res"] = torch.empty((T, H), dtype=dt, device=dev) if case["y"] else None
            s["normed"] = torch.empty((T, H), dtype=dt, device=dev)
            return s
        # what the forward pass stored as res, and the gradients that come back
        s["res"] = x.to(dt)
        s["dnormed"], s["dres"] = _normal(gen, (T, H), dt), _normal(gen, (T, H), dt)
        s["dx"] = torch.empty((T, H), dtype=dt, device=dev)
        s["dw_pre"] = torch.empty((H,), dtype=torch.float32, device=dev)
        s["dy"] = torch.empty((T, H), dtype=dt, device=dev) if case["y"] else None
        s["dw_post"] = torch.empty((H,), dtype=torch.float32, device=dev) if case["post"] else None
        s["dgate"] = torch.empty((T,), dtype=torch.float32, device=dev) if case["gate"] else None
        return s
    I = case["I"]
    s["x"] = _normal(gen, (T, H), dt)
    s["w13"] = _normal(gen, (2 * I, H), dt, 1.5 * H ** -0.5)
    s["w2"] = _normal(gen, (H, I), dt, I ** -0.5)
    s["out"] = torch.empty((T, H), dtype=dt, device=dev)
    s["base"] = _normal(gen, (T, H), dt) if case["base"] else None
    if case["grad"]:
        s["dout"] = _normal(gen, (T, H), dt)
        s["dx"] = torch.empty((T, H), dtype=dt, device=dev)
        s["dw13"] = torch.empty((2 * I, H), dtype=dt, device=dev)
        s["dw2"] = torch.empty((H, I), dtype=dt, device=dev)
    if case["op"] == "keep8":
        s["x8"], s["x8_scale"] = _mx_rows(s["x"])
        s["kept"] = torch.empty((T, 2 * I), dtype=torch.uint8, device=dev)
        s["kept_scale"] = torch.empty((T, 2 * I // 32), dtype=torch.uint8, device=dev)
    elif case["grad"]:
        s["kept"] = torch.empty((T, 2 * I), dtype=dt, device=dev)
    return s


# ---- one pass --------------------------------------------------------------------------


def _plan(s):
    """The shape (and workspace) that a program keeps for its calls."""
    import dispatch_grouped_gemm_amd as moe
    c = s["case"]
    if c["op"] == "norm":
        shape = moe.NormShape(T=c["T"], H=c["H"], eps=EPS, skip_scale=c["skip"],
                              block_scale=c["scale"])
        ws = moe.alloc_norm_workspace(shape, _device()) if c["grad"] else None
    else:
        shape = moe.FfnShape(T=c["T"], H=c["H"], I=c["I"], gate_limit=c["limit"],
                             up_limit=c["limit"])
        ws = moe.alloc_ffn_workspace(shape, _device(), backward=c["grad"])
    s["plan"] = moe, shape, ws
    return s["plan"]


def _run_own(s):
    c = s["case"]
    moe, shape, ws = s.get("plan") or _plan(s)
    if c["op"] == "norm":
        if not c["grad"]:
            moe.moe_norm_forward(shape, s["x"], s["w_pre"], s["normed"], y=s["y"],
                                 w_post=s["w_post"], gate=s["gate"], res=s["res"])
            return [t for t in (s["res"], s["normed"]) if t is not None]
        moe.moe_norm_backward(shape, s["dnormed"], s["res"], s["w_pre"], s["dx"], s["dw_pre"], ws,
                              dres=s["dres"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                              dy=s["dy"], dw_post=s["dw_post"], dgate=s["dgate"])
        return [t for t in (s["dx"], s["dw_pre"], s["dy"], s["dw_post"], s["dgate"])
                if t is not None]
    kept, scale = s.get("kept"), s.get("kept_scale")
    moe.moe_ffn_forward(shape, s["x"], s["w13"], s["w2"], s["out"], ws, base=s["base"],
                        gate_up=kept, gate_up_scale=scale)
    if not c["grad"]:
        return [s["out"]]
    eight = c["op"] == "keep8"
    moe.moe_ffn_backward(shape, s["dout"], s["x8"] if eight else s["x"], s["w13"], s["w2"], kept,
                         s["dx"], s["dw13"], s["dw2"], ws, gate_up_scale=scale,
                         x_scale=s["x8_scale"] if eight else None)
    grads = [s["out"], s["dx"], s["dw13"], s["dw2"]]
    return grads if eight else grads + [kept]


def _mx_values(codes, scale):
    """float32 values of MX FP8 rows."""
    v = codes.view(torch.float8_e4m3fn).float().reshape(codes.shape[0], -1, 32)
    return torch.ldexp(v, scale.to(torch.int32)[:, :, None] - 127).reshape(codes.shape)


def _plain_norm(s):
    c = s["case"]
    w_pre = s["w_pre"].float()
    if not c["grad"]:
        dt = s["x"].dtype
        r = s["x"].float()
        if c["y"]:
            z = s["y"].float()
            if c["post"]:
                z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["w_post"].float()
            z = z * c["scale"]
            if c["gate"]:
                z = z * torch.sigmoid(s["gate"])[:, None]
            r = c["skip"] * r + z
        res = r.to(dt)
        # the norm is of what is stored
        r = res.float()
        n = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * w_pre
        return [res, n.to(dt)] if c["y"] else [n.to(dt)]
    dt = s["res"].dtype
    r, dn = s["res"].float(), s["dnormed"].float()
    rho = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    hat, g = r * rho, dn * w_pre
    dr = s["dres"].float() + rho * (g - hat * (g * hat).mean(1, keepdim=True))
    dw_pre = (dn * hat).sum(0)
    if not c["y"]:
        return [dr.to(dt), dw_pre]
    y, f = s["y"].float(), c["scale"]
    if c["gate"]:
        sig = torch.sigmoid(s["gate"])[:, None]
        f = f * sig
    outs = [(c["skip"] * dr).to(dt), dw_pre]
    z, dz = y, dr * f
    if c["post"]:
        rho = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
        hat, w = y * rho, s["w_post"].float()
        z, g = hat * w, dz * w
        outs += [(rho * (g - hat * (g * hat).mean(1, keepdim=True))).to(dt), (dz * hat).sum(0)]
    else:
        outs += [dz.to(dt)]
    if c["gate"]:
        outs += [(dr * z).sum(1) * (c["scale"] * sig * (1.0 - sig))[:, 0]]
    return outs


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s)
    I, lim, dt = c["I"], c["limit"], s["x"].dtype
    w13, w2 = s["w13"].float(), s["w2"].float()
    gu = s["x"].float() @ w13.t()
    g, u = gu[:, :I].clamp(max=lim), gu[:, I:].clamp(-lim, lim)
    out = (g * torch.sigmoid(g) * u) @ w2.t()
    if s["base"] is not None:
        out = out + s["base"].float()
    out = out.to(dt)
    if not c["grad"]:
        return [out]
    # the backward pass has what was kept: rounded to the type, or to 8 bits
    if c["op"] == "keep8":
        x, gu = _mx_values(s["x8"], s["x8_scale"]), _mx_values(*_mx_rows(gu))
    else:
        x, kept = s["x"].float(), gu.to(dt)
        gu = kept.float()
    dout = s["dout"].float()
    g, u = gu[:, :I].clamp(max=lim), gu[:, I:].clamp(-lim, lim)
    sig = torch.sigmoid(g)
    dh = dout @ w2
    dg = torch.where(gu[:, :I] > lim, 0.0, dh * u * sig * (1.0 + g * (1.0 - sig)))
    du = torch.where(gu[:, I:].abs() > lim, 0.0, dh * g * sig)
    d = torch.cat([dg, du], 1)
    grads = [out, (d @ w13).to(dt), (d.t() @ x).to(dt), (dout.t() @ (g * sig * u)).to(dt)]
    return grads if c["op"] == "keep8" else grads + [kept]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------------


def work(case):
    T, H, b = case["T"], case["H"], BYTES[case["dtype"]]
    if case["op"] == "norm":
        rows = T * H * b
        if not case["grad"]:
            # x in and normed out; with a block its output in and res out
            n = 4 if case["y"] else 2
            return dict(bytes=n * rows + H * b * (1 + case["post"]) + 4 * T * case["gate"],
                        flops=T * H * (4 + 4 * case["y"] + 4 * case["post"]))
        # dnormed, dres and res in, dx out; with a block its output in and dy out
        n = 6 if case["y"] else 4
        return dict(bytes=n * rows + H * (b + 4) * (1 + case["post"]) + 8 * T * case["gate"],
                    flops=T * H * (10 + 6 * case["y"] + 10 * case["post"]))
    I = case["I"]
    one, weights = T * H * b, 3 * H * I * b
    byt, flops = 2 * one + weights + (one if case["base"] else 0), 6 * T * H * I
    if case["grad"]:
        # dout in, dx and the weights' gradients out, and what is kept
        kept = T * 2 * I * 33 / 32 + T * H * 33 / 32 if case["op"] == "keep8" else T * 2 * I * b
        byt += 2 * one + weights + kept
        flops += 12 * T * H * I
    return dict(bytes=byt, flops=flops)


# ---- the definition in 64 bits ---------------------------------------------------------


def _exact_mx(v):
    """v as MX FP8 holds it: 4 significant bits, at least 2^-9 of the block's power."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 8)
    a = (b / unit).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(a / step) * step * unit).reshape(v.shape)


def _exact_rms(v):
    return 1.0 / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)


def _exact_rms_back(v, d):
    """The gradient of v / sqrt(mean v^2 + eps) for that of the result."""
    q = _exact_rms(v)
    return q * d - v * q ** 3 * (v * d).sum(1, keepdim=True) / v.shape[1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        w = s["w_pre"].double()
        a = torch.full((case["T"], 1), case["scale"], dtype=torch.float64, device=w.device)
        p = None
        if case["gate"]:
            p = 1.0 / (1.0 + torch.exp(-s["gate"].double()[:, None]))
            a = a * p
        y = s["y"].double() if case["y"] else None
        z = y
        if case["post"]:
            z = y * _exact_rms(y) * s["w_post"].double()
        if not case["grad"]:
            r = s["x"].double()
            if case["y"]:
                r = r * case["skip"] + a * z
            stored = r.to(s["x"].dtype).double()
            n = stored * _exact_rms(stored) * w
            return [r, n] if case["y"] else [n]
        r, dn = s["res"].double(), s["dnormed"].double()
        dr = s["dres"].double() + _exact_rms_back(r, dn * w)
        outs = [dr * (case["skip"] if case["y"] else 1.0), (dn * r * _exact_rms(r)).sum(0)]
        if case["post"]:
            outs += [_exact_rms_back(y, a * dr * s["w_post"].double()),
                     (a * dr * y * _exact_rms(y)).sum(0)]
        elif case["y"]:
            outs += [a * dr]
        if case["gate"]:
            outs += [(dr * z).sum(1) * case["scale"] * (p * (1.0 - p))[:, 0]]
        return outs
    I, lim, dt = case["I"], case["limit"], s["x"].dtype
    x, w13, w2 = s["x"].double(), s["w13"].double(), s["w2"].double()
    g, u = x @ w13[:I].t(), x @ w13[I:].t()
    top = torch.full((), lim, dtype=torch.float64, device=x.device)

    def act(g):
        m = torch.minimum(g, top)
        return m / (1.0 + torch.exp(-m))

    def cut(u):
        return torch.maximum(torch.minimum(u, top), -top)

    out = (act(g) * cut(u)) @ w2.t()
    if case["base"]:
        out = out + s["base"].double()
    if not case["grad"]:
        return [out]
    kept = torch.cat([g, u], 1)
    if case["op"] == "keep8":
        gu, x = _exact_mx(kept), _exact_mx(x)
    else:
        gu = kept.to(dt).double()
    g, u = gu[:, :I], gu[:, I:]
    dout = s["dout"].double()
    dh = dout @ w2
    e = torch.exp(-torch.minimum(g, top))
    slope = 1.0 / (1.0 + e) + torch.minimum(g, top) * e / (1.0 + e) ** 2
    dg = dh * cut(u) * slope * (g <= top)
    du = dh * act(g) * (u.abs() <= top)
    grads = [out, dg @ w13[:I] + du @ w13[I:], torch.cat([dg.t() @ x, du.t() @ x]),
             dout.t() @ (act(g) * cut(u))]
    return grads if case["op"] == "keep8" else grads + [kept]
