"""What is measured of the operators around the scan: the short causal convolution, the selective scan
and the gated group norm, each on the paths that use it (prompt, single tokens, training).

``run`` computes a pass either in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, with ``own`` true, by the library's entry points.  Inputs are laid out as a layer has
them: the convolution's input and the gate are slices of one projection, B and C of the scan are slices
of another, so they come with a token stride of their own.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # prompt of a 2.7B layer: the x, B, C slice (5120 + 2 x 128) of a projection of width 10576
        {"name": "conv prompt", "op": "conv_fwd", "batch": 2, "len": 8192, "ch": 5120, "side": 128, "pad": 5200,
         "width": 4, "init": False, "dtype": "bf16"},
        # the same layer in training
        {"name": "conv train", "op": "conv_bwd", "batch": 2, "len": 4096, "ch": 5120, "side": 128, "pad": 5200,
         "width": 4, "init": False, "dtype": "bf16"},
        # one token for each of 128 requests
        {"name": "conv decode", "op": "conv_step", "batch": 128, "len": 1, "ch": 5120, "side": 128, "pad": 5200,
         "width": 4, "init": True, "dtype": "bf16"},
        # a continued prompt in fp32 whose sizes fit no vector
        {"name": "conv odd", "op": "conv_fwd", "batch": 3, "len": 1021, "ch": 777, "side": 0, "pad": 0,
         "width": 3, "init": True, "dtype": "fp32"},
        # one prompt of 2048 tokens, 5120 channels of 16 states, with the gate
        {"name": "scan prompt", "op": "scan_fwd", "batch": 1, "len": 2048, "ch": 5120, "state": 16, "groups": 1,
         "gate": True, "init": False, "dtype": "bf16"},
        # continued fp32 prompts, ragged in every size, no gate
        {"name": "scan odd", "op": "scan_fwd", "batch": 3, "len": 701, "ch": 1111, "state": 19, "groups": 1,
         "gate": False, "init": True, "dtype": "fp32"},
        # one token for each of 128 requests
        {"name": "scan decode", "op": "scan_step", "batch": 128, "len": 1, "ch": 5120, "state": 16, "groups": 1,
         "gate": True, "init": True, "dtype": "bf16"},
        # a training step's backward pass
        {"name": "scan train", "op": "scan_bwd", "batch": 2, "len": 2048, "ch": 5120, "state": 16, "groups": 1,
         "gate": True, "init": False, "dtype": "bf16"},
        # a small fp32 model with two groups of B and C and no gate
        {"name": "scan train odd", "op": "scan_bwd", "batch": 2, "len": 515, "ch": 770, "state": 16, "groups": 2,
         "gate": False, "init": True, "dtype": "fp32"},
        # the layer's output norm over a prompt
        {"name": "norm prompt", "op": "norm_fwd", "batch": 2, "len": 8192, "ch": 5120, "groups": 1, "pad": 5456,
         "before": False, "dtype": "bf16"},
        # the same in training, eight groups of 512 channels
        {"name": "norm train", "op": "norm_bwd", "batch": 2, "len": 4096, "ch": 4096, "groups": 8, "pad": 0,
         "before": False, "dtype": "bf16"},
        # one token of one request: the smallest call
        {"name": "norm one token", "op": "norm_fwd", "batch": 1, "len": 1, "ch": 5120, "groups": 1, "pad": 5456,
         "before": False, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    case = {"op": op, "dtype": dtype}
    batch = _spread(rng, 1, 192) if op.endswith("step") else _spread(rng, 1, 8)
    length = rng.randint(1, 4) if op.endswith("step") else _spread(rng, 1, 8192)
    ch = _spread(rng, 16, 8192)
    if rng.random() < 0.6:
        ch = 8 * max(2, ch // 8)    # most widths are whole vectors, some are not
    if op.startswith("conv"):
        side = rng.choice([0, 16, 64, 128, 256])
        most = 2 * 8192 * 5376 if op == "conv_fwd" else 2 * 4096 * 5376
        case.update(side=side, pad=rng.choice([0, 1, 8, 24, 2048]), width=rng.randint(2, 4),
                    init=op == "conv_step" or rng.random() < 0.5)
        length = max(1, min(length, most // (batch * (ch + 2 * side) * (2 if dtype == "fp32" else 1))))
    elif op.startswith("scan"):
        state = rng.choice([4, 8, 16, 16, 16, 32, 64, rng.randint(1, 64)])
        groups = rng.choice([1, 1, 2]) if ch % 2 == 0 else 1
        most = {"scan_fwd": 2048 * 5120 * 16, "scan_bwd": 2 * 2048 * 5120 * 16, "scan_step": 128 * 5120 * 16}[op]
        case.update(state=state, groups=groups, gate=rng.random() < 0.6,
                    init=op == "scan_step" or rng.random() < 0.5)
        if op == "scan_step":
            batch = max(1, min(batch, most // (ch * state * length)))
        else:
            length = max(1, min(length, most // (batch * ch * state)))
    else:
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if ch % g == 0])
        most = 2 * 8192 * 5120 if op == "norm_fwd" else 2 * 4096 * 4096
        case.update(groups=groups, pad=rng.choice([0, 1, 8, 336]), before=rng.random() < 0.3)
        length = max(1, min(length, most // (batch * ch * (2 if dtype == "fp32" else 1))))
    case.update(batch=batch, len=length, ch=ch)
    return case


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g, io = _gen(seed), _DTYPES[case["dtype"]]
    bsz, length, ch = case["batch"], case["len"], case["ch"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case)
    if case["op"].startswith("conv"):
        total, width = ch + 2 * case["side"], case["width"]
        rows = normal(bsz, length, case["pad"] + total, dtype=io)
        s["x"] = rows[:, :, case["pad"]:]
        s["split"] = (ch, case["side"], case["side"]) if case["side"] else None
        s["w"] = (torch.rand(total, width, generator=g, device="cuda") * 2 - 1) / math.sqrt(width)
        s["bias"] = normal(total, std=0.1)
        s["init"] = normal(bsz, width - 1, total, dtype=io) if case["init"] else None
        if case["op"] == "conv_bwd":
            s["dy"] = [normal(bsz, length, n, dtype=io) for n in (s["split"] or (total,))]
    elif case["op"].startswith("scan"):
        n, groups = case["state"], case["groups"]
        s["x"] = torch.nn.functional.silu(normal(bsz, length, ch)).to(io)
        step = torch.exp(torch.rand(ch, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["dt"] = normal(bsz, length, ch, std=0.5, dtype=io)
        s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(ch, n, std=0.1))
        s["D"] = normal(ch)
        rank = max(1, ch // 16)
        rows = normal(bsz, length, rank + 2 * groups * n, std=1.0 / math.sqrt(n), dtype=io)
        s["B"] = rows[:, :, rank:rank + groups * n].unflatten(2, (groups, n))
        s["C"] = rows[:, :, rank + groups * n:].unflatten(2, (groups, n))
        s["z"] = normal(bsz, length, 2 * ch, dtype=io)[:, :, ch:] if case["gate"] else None
        s["init"] = normal(bsz, ch, n, std=0.1) if case["init"] else None
        if case["op"] == "scan_bwd":
            s["dy"] = normal(bsz, length, ch, dtype=io)
            s["dfinal"] = normal(bsz, ch, n, std=0.1) if case["init"] else None
    else:
        s["x"] = normal(bsz, length, ch, dtype=io)
        s["z"] = normal(bsz, length, ch + case["pad"], dtype=io)[:, :, :ch]
        s["w"] = 1.0 + normal(ch, std=0.1)
        if case["op"] == "norm_bwd":
            s["dy"] = normal(bsz, length, ch, dtype=io)
    return s


def run(s):
    if own:
        return _own(s)
    return {"conv_fwd": _conv_fwd, "conv_step": _conv_step, "conv_bwd": _conv_bwd, "scan_fwd": _scan_fwd,
            "scan_step": _scan_step, "scan_bwd": _scan_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}[s["op"]](s)


def _own(s):
    import state_space_sequence_03_amd as ssd
    op = s["op"]
    if op == "conv_fwd":
        y, fin = ssd.ssd_conv_fwd(s["x"], s["w"], s["bias"], s["init"], split=s["split"], want_final_state=True)
        return {"y": y, "final": fin}
    if op == "conv_step":
        y = ssd.ssd_conv_step(s["init"], s["x"], s["w"], s["bias"], split=s["split"])
        return {"y": y, "state": s["init"]}
    if op == "conv_bwd":
        dy = tuple(s["dy"]) if s["split"] else s["dy"][0]
        got = ssd.ssd_conv_bwd(s["x"], s["w"], s["bias"], s["init"], dy, want_dinit=s["init"] is not None)
        return {k: got[k] for k in ("dx", "dweight", "dbias", "dinit")}
    if op == "scan_fwd":
        y, fin = ssd.ssd_selscan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["init"],
                                     dt_bias=s["dt_bias"], dt_softplus=True)
        return {"y": y, "final": fin}
    if op == "scan_step":
        y = ssd.ssd_selscan_step(s["init"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                 dt_bias=s["dt_bias"], dt_softplus=True)
        return {"y": y, "state": s["init"]}
    if op == "scan_bwd":
        got = ssd.ssd_selscan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["init"], s["dy"], s["dfinal"],
                                  dt_bias=s["dt_bias"], dt_softplus=True, want_dinit=s["init"] is not None,
                                  want_ddt_bias=True)
        return {k: got[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dinit", "ddt_bias")}
    if op == "norm_fwd":
        return ssd.ssd_gated_norm_fwd(s["x"], s["z"], s["w"], ngroups=s["groups"], norm_before_gate=s["before"])
    got = ssd.ssd_gated_norm_bwd(s["x"], s["z"], s["w"], s["dy"], ngroups=s["groups"], norm_before_gate=s["before"])
    return {k: got[k] for k in ("dx", "dz", "dweight")}


# ---- the plain forms ----

def _zero_window(s):
    bsz, _, total = s["x"].shape
    return torch.zeros(bsz, s["width"] - 1, total, device="cuda", dtype=s["x"].dtype)


def _window(s):
    """The inputs with the W - 1 earlier ones in front."""
    return torch.cat([_zero_window(s) if s["init"] is None else s["init"], s["x"]], 1)


def _shifted(full, length, w):
    """sum_k w[:, k] full[:, t + k] over the width."""
    return sum(full[:, k:k + length].float() * w[:, k] for k in range(w.shape[1]))


def _parts(y, split):
    return [p.contiguous() for p in y.split(split, 2)] if split else y


def _conv_fwd(s):
    full, length = _window(s), s["x"].shape[1]
    u = _shifted(full, length, s["w"]) + s["bias"]
    y = (u * torch.sigmoid(u)).to(s["x"].dtype)
    return {"y": _parts(y, s["split"]), "final": full[:, length:].contiguous()}


def _conv_step(s):
    got = _conv_fwd(s)
    s["init"].copy_(got["final"])
    return {"y": got["y"], "state": s["init"]}


def _conv_bwd(s):
    full, length, w = _window(s), s["x"].shape[1], s["w"]
    width = w.shape[1]
    u = _shifted(full, length, w) + s["bias"]
    sg = torch.sigmoid(u)
    du = torch.cat(s["dy"], 2).float() * (sg * (1 + u * (1 - sg)))
    dw = torch.stack([(du * full[:, k:k + length].float()).sum((0, 1)) for k in range(width)], 1)
    room = torch.nn.functional.pad(du, (0, 0, width - 1, width - 1))
    dfull = _shifted(room, length + width - 1, w.flip(1)).to(s["x"].dtype)
    return {"dx": dfull[:, width - 1:].contiguous(), "dweight": dw, "dbias": du.sum((0, 1)),
            "dinit": dfull[:, :width - 1].contiguous() if s["init"] is not None else None}


def _prepared(s):
    """Step sizes, decays [B, L, D, N], and B and C spread over the channels of their group."""
    raw = s["dt"].float() + s["dt_bias"]
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    a = torch.exp(dt.unsqueeze(3) * s["A"])
    per = s["ch"] // s["groups"]
    return raw, dt, a, s["B"].float().repeat_interleave(per, 2), s["C"].float().repeat_interleave(per, 2)


def _linear_scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along axis 1, from zero, in log2(L) doublings (both arguments are used up)."""
    d, length = 1, a.shape[1]
    while d < length:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _states(s, a, dt, x, bb):
    b = (dt * x).unsqueeze(3) * bb
    if s["init"] is not None:
        b[:, 0] += a[:, 0] * s["init"]
    return _linear_scan(a, b)


def _scan_fwd(s):
    _, dt, a, bb, cc = _prepared(s)
    x = s["x"].float()
    h = _states(s, a, dt, x, bb)
    y = (h * cc).sum(3) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return {"y": y.to(s["x"].dtype), "final": h[:, -1].contiguous()}


def _scan_step(s):
    got = _scan_fwd(s)
    s["init"].copy_(got["final"])
    return {"y": got["y"], "state": s["init"]}


def _scan_bwd(s):
    io, per = s["x"].dtype, s["ch"] // s["groups"]
    raw, dt, a, bb, cc = _prepared(s)
    x, dy = s["x"].float(), s["dy"].float()
    h = _states(s, a, dt, x, bb)
    dz = None
    ds = dy
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        ds = dy * z * sg
        dz = (dy * ((h * cc).sum(3) + s["D"] * x) * (sg * (1 + z * (1 - sg)))).to(io)
    first = s["init"].unsqueeze(1) if s["init"] is not None else torch.zeros_like(h[:, :1])
    before = torch.cat([first, h[:, :-1]], 1)
    from_y = ds.unsqueeze(3) * cc
    if s["dfinal"] is not None:
        from_y[:, -1] += s["dfinal"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _linear_scan(later.flip(1), from_y.flip(1)).flip(1)
    del later, from_y
    group = lambda t: t.unflatten(2, (s["groups"], per)).sum(3).to(io)
    dcc, dbb = group(h * ds.unsqueeze(3)), group(g * (dt * x).unsqueeze(3))
    dinit = (a[:, 0] * g[:, 0]) if s["init"] is not None else None
    q = (g * bb).sum(3)
    flow = g * a * before
    ddt = (x * q + (flow * s["A"]).sum(3)) * torch.sigmoid(raw)
    return {"dx": (dt * q + s["D"] * ds).to(io), "ddt": ddt.to(io), "dA": (flow * dt.unsqueeze(3)).sum((0, 1)),
            "dB": dbb, "dC": dcc, "dD": (ds * x).sum((0, 1)), "dz": dz, "dinit": dinit, "ddt_bias": ddt.sum((0, 1))}


def _grouped(s, t):
    return t.unflatten(-1, (s["groups"], -1))


def _norm_fwd(s, eps=1e-5):
    x, z = s["x"].float(), s["z"].float()
    gate = z * torch.sigmoid(z)
    u = _grouped(s, x if s["before"] else x * gate)
    n = (u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps)).flatten(-2) * s["w"]
    return (n * gate if s["before"] else n).to(s["x"].dtype)


def _norm_bwd(s, eps=1e-5):
    io, x, z, dy = s["x"].dtype, s["x"].float(), s["z"].float(), s["dy"].float()
    sg = torch.sigmoid(z)
    gate, dgate = z * sg, sg * (1 + z * (1 - sg))
    u = _grouped(s, x if s["before"] else x * gate)
    r = torch.rsqrt(u.square().mean(-1, keepdim=True) + eps)
    n = (u * r).flatten(-2)
    dn = dy * gate if s["before"] else dy
    dw = (dn * n).sum((0, 1))
    t = _grouped(s, dn * s["w"])
    du = (r * t - u * (r * r * r) * (t * u).mean(-1, keepdim=True)).flatten(-2)
    if s["before"]:
        return {"dx": du.to(io), "dz": (dy * n * s["w"] * dgate).to(io), "dweight": dw}
    return {"dx": (du * gate).to(io), "dz": (du * x * dgate).to(io), "dweight": dw}


# ---- what cannot be done without ----

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows, ch = case["batch"] * case["len"], case["ch"]
    if case["op"].startswith("conv"):
        total, width = ch + 2 * case["side"], case["width"]
        cells, window = rows * total, case["batch"] * (width - 1) * total
        params = 4 * total * (width + 1)
        if case["op"] == "conv_bwd":
            return {"bytes": 3 * e * cells + (2 * e * window if case["init"] else 0) + 2 * params,
                    "flops": cells * (6 * width + 14)}
        return {"bytes": 2 * e * cells + e * window * (2 if case["init"] else 1) + params,
                "flops": cells * (2 * width + 6)}
    if case["op"].startswith("scan"):
        n, cells = case["state"], rows * ch
        state, bc = 4 * case["batch"] * ch * n, 2 * e * rows * case["groups"] * n
        params = 4 * ch * (n + 2)
        if case["op"] == "scan_bwd":
            return {"bytes": e * cells * (7 if case["gate"] else 5) + 2 * bc + (3 * state if case["init"] else 0) + 2 * params,
                    "flops": cells * (26 * n + 40)}
        return {"bytes": e * cells * (4 if case["gate"] else 3) + bc + state * (2 if case["init"] else 1) + params,
                "flops": cells * (7 * n + 20)}
    if case["op"] == "norm_bwd":
        return {"bytes": 5 * e * rows * ch + 8 * ch, "flops": 30 * rows * ch}
    return {"bytes": 3 * e * rows * ch + 4 * ch, "flops": 12 * rows * ch}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        if case["op"].startswith("scan"):
            return _exact_scan(s)
    return (_exact_conv if case["op"].startswith("conv") else _exact_norm)(s)


def _leaf(t):
    return t.detach().double().requires_grad_(True)


def _exact_conv(s):
    bsz, length, total = s["x"].shape
    width = s["width"]
    x, w, bias = _leaf(s["x"]), _leaf(s["w"]), _leaf(s["bias"])
    init = _leaf(s["init"]) if s["init"] is not None else torch.zeros(bsz, width - 1, total, device="cuda", dtype=torch.float64)
    full = torch.cat([init, x], 1)
    with torch.set_grad_enabled(s["op"] == "conv_bwd"):
        u = bias + torch.zeros(bsz, length, total, device="cuda", dtype=torch.float64)
        for k in range(width):
            u = u + full.narrow(1, k, length) * w.select(1, k)
        y = u / (1 + torch.exp(-u))
    cut = s["split"] or (total,)
    if s["op"] != "conv_bwd":
        ys = list(torch.split(y.detach(), cut, 2))
        last = full.detach()[:, full.shape[1] - (width - 1):].contiguous()
        if s["op"] == "conv_step":
            return {"y": ys if s["split"] else ys[0], "state": last}
        return {"y": ys if s["split"] else ys[0], "final": last}
    y.backward(torch.cat([d.double() for d in s["dy"]], 2))
    return {"dx": x.grad, "dweight": w.grad, "dbias": bias.grad, "dinit": init.grad if s["init"] is not None else None}


def _exact_norm(s, eps=1e-5):
    x, z, w = _leaf(s["x"]), _leaf(s["z"]), _leaf(s["w"])
    with torch.set_grad_enabled(s["op"] == "norm_bwd"):
        gate = z / (1 + torch.exp(-z))
        v = x if s["before"] else x * gate
        shape = v.shape
        v = v.reshape(shape[0], shape[1], s["groups"], -1)
        v = (v / torch.sqrt((v * v).sum(-1, keepdim=True) / v.shape[-1] + eps)).reshape(shape) * w
        y = v * gate if s["before"] else v
    if s["op"] == "norm_fwd":
        return y.detach()
    y.backward(s["dy"].double())
    return {"dx": x.grad, "dz": z.grad, "dweight": w.grad}


def _exact_scan(s):
    """The recurrence token by token, and its derivative from the last token to the first."""
    f = lambda t: t.double() if t is not None else None
    x, A, D, z = f(s["x"]), f(s["A"]), f(s["D"]), f(s["z"])
    bsz, length, ch = x.shape
    which = torch.arange(ch, device="cuda") // (ch // s["groups"])
    raw = f(s["dt"]) + f(s["dt_bias"])
    dt = torch.log1p(torch.exp(raw))
    dt = torch.where(torch.isinf(dt), raw, dt)
    h = f(s["init"]).clone() if s["init"] is not None else torch.zeros(bsz, ch, A.shape[1], device="cuda", dtype=torch.float64)
    back = s["op"] == "scan_bwd"
    kept = [h] if back else None
    y = torch.empty_like(x)
    for t in range(length):
        bt, ct = f(s["B"][:, t])[:, which], f(s["C"][:, t])[:, which]
        h = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[:, :, None] * bt
        y[:, t] = (h * ct).sum(2)
        if back:
            kept.append(h)
    y = y + D * x
    if not back:
        out = y if z is None else y * z / (1 + torch.exp(-z))
        return {"y": out, "state" if s["op"] == "scan_step" else "final": h}
    dy = f(s["dy"])
    sg = 1 / (1 + torch.exp(-z)) if z is not None else None
    ds = dy if z is None else dy * z * sg
    g = f(s["dfinal"]).clone() if s["dfinal"] is not None else torch.zeros_like(h)
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dA = torch.zeros_like(A)
    dB = torch.zeros(bsz, length, s["groups"], A.shape[1], device="cuda", dtype=torch.float64)
    dC = torch.zeros_like(dB)
    for t in range(length - 1, -1, -1):
        bt, ct = f(s["B"][:, t])[:, which], f(s["C"][:, t])[:, which]
        g = g + ds[:, t, :, None] * ct
        a = torch.exp(dt[:, t, :, None] * A)
        dC[:, t] = (ds[:, t, :, None] * kept[t + 1]).reshape(bsz, s["groups"], -1, A.shape[1]).sum(2)
        dB[:, t] = (g * (dt[:, t] * x[:, t])[:, :, None]).reshape(bsz, s["groups"], -1, A.shape[1]).sum(2)
        q = (g * bt).sum(2)
        flow = g * a * kept[t]
        dx[:, t] = dt[:, t] * q + D * ds[:, t]
        ddt[:, t] = x[:, t] * q + (flow * A).sum(2)
        dA += (flow * dt[:, t, :, None]).sum(0)
        g = g * a
    ddt = ddt / (1 + torch.exp(-raw))
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (ds * x).sum((0, 1)),
            "dz": dy * y * sg * (1 + z * (1 - sg)) if z is not None else None,
            "dinit": g if s["init"] is not None else None, "ddt_bias": ddt.sum((0, 1))}
