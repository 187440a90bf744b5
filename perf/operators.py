"""What is measured of the operators around the convolution layers: group norm
with an activation (channels last, forward and gradient), the loss of a class
head over many classes (with its gradient, the logits never stored) and the
pointwise layer with 4-bit weights that answers with such a head.

Each case runs in two forms that take the same inputs: a plain one in
elementary torch operations and 32 bits, rounded once at the end, and, where
``own`` is true, this package's entry points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_MOST_GN = 16 * 160 * 160 * 128          # elements of the largest feature map
_MOST_LOSS = 8192 * 1024 * 65536         # rows x features x classes of the largest loss
_MOST_W4 = 8192 * 28672                  # weights of the largest 4-bit layer


# ------------------------------------------------------------------ the cases
def _gn(name, n, h, w, c, groups, dtype, act, grad, wide=0):
    return {"name": name, "op": "group_norm", "n": n, "h": h, "w": w, "c": c, "groups": groups, "dtype": dtype,
            "act": act, "grad": grad, "wide": wide}


def _loss(name, rows, features, classes, grad):
    return {"name": name, "op": "class_loss", "rows": rows, "features": features, "classes": classes, "grad": grad}


def _w4(name, rows, c_in, c_out, group, dtype, act):
    return {"name": name, "op": "w4", "rows": rows, "c_in": c_in, "c_out": c_out, "group": group, "dtype": dtype,
            "act": act}


def listed():
    return [
        # the last stage of a small classifier, one image: only latency counts
        _gn("gn_7x7x512_b1_bf16", 1, 7, 7, 512, 32, "bf16", "relu", False),
        # after the batch-8 3x3 256->256 layer of the throughput sweep
        _gn("gn_80x80x256_b8_bf16", 8, 80, 80, 256, 32, "bf16", "mish", False),
        # a training batch in fp32, larger than the L2
        _gn("gn_160x160x128_b16_f32", 16, 160, 160, 128, 32, "f32", "mish", False),
        # keyword-spotting sized, ragged groups of ten channels, with the gradient
        _gn("gn_grad_25x5x60_b3_f32", 3, 25, 5, 60, 6, "f32", "relu", True),
        # the sweep's layer in training
        _gn("gn_grad_80x80x256_b8_bf16", 8, 80, 80, 256, 32, "bf16", "mish", True),
        # a channel slice of a concatenated buffer, in training
        _gn("gn_grad_slice_40x40x512_b8_bf16", 8, 40, 40, 512, 16, "bf16", "mish", True, 512),
        # a thousand classes, a handful of images
        _loss("loss_grad_20x512x1000", 20, 512, 1000, True),
        # evaluation of one 40x40 map over an odd number of classes
        _loss("loss_1600x1024x32003", 1600, 1024, 32003, False),
        # a training batch over a large vocabulary
        _loss("loss_grad_8192x1024x65536", 8192, 1024, 65536, True),
        # one pooled feature vector to a thousand classes: latency
        _w4("w4_1x1024x1000_bf16", 1, 1024, 1000, 128, "bf16", "none"),
        # one row through a wide layer: the weights' bytes
        _w4("w4_1x8192x28672_bf16", 1, 8192, 28672, 128, "bf16", "mish"),
        # ragged sizes, fine groups, several rows, fp32 activations
        _w4("w4_13x2047x5001_f32", 13, 2047, 5001, 32, "f32", "relu"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group_norm", "group_norm", "class_loss", "w4"])
    if op == "group_norm":
        groups = rng.choice([1, 2, 3, 4, 6, 8, 16, 32])
        while True:
            c = groups * _log(rng, 1, 96)
            n, h, w = _log(rng, 1, 16), _log(rng, 1, 160), _log(rng, 1, 160)
            if c <= 1024 and n * h * w * c <= _MOST_GN and h * w * (c // groups) >= 8:
                break
        case = _gn("", n, h, w, c, groups, rng.choice(["bf16", "f32"]), rng.choice(["none", "relu", "mish"]),
                   rng.random() < 0.5, rng.choice([0, 0, c]))
    elif op == "class_loss":
        while True:
            rows, features, classes = _log(rng, 1, 8192), _log(rng, 32, 2048), _log(rng, 200, 65536)
            if rng.random() < 0.7:
                features = -(-features // 8) * 8
            if rows * features * classes <= _MOST_LOSS:
                break
        case = _loss("", rows, features, classes, rng.random() < 0.7)
    else:
        while True:
            c_in, c_out = _log(rng, 64, 8192), _log(rng, 64, 28672)
            if rng.random() < 0.5:
                c_in = -(-c_in // 64) * 64
            if c_in * c_out <= _MOST_W4:
                break
        case = _w4("", _log(rng, 1, 64), c_in, c_out, rng.choice([32, 64, 128]), rng.choice(["bf16", "f32"]),
                   rng.choice(["none", "relu", "mish"]))
    del case["name"]
    return case


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(case, seed):
    g = _generator(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {}
    if case["op"] == "group_norm":
        n, h, w, c, dt = case["n"], case["h"], case["w"], case["c"], _DT[case["dtype"]]
        # a convolution's output before its normalisation: channels of their own mean and spread
        spread, mean = 0.5 + torch.rand(c, generator=g, device="cuda"), 0.5 + randn(c)

        def maps(scale, shift):
            buf = torch.empty(n, h, w, c + case["wide"], device="cuda", dtype=dt)
            view = buf[..., case["wide"]:]
            view.copy_(randn(n, h, w, c) * scale + shift)
            return view

        s["x"] = maps(spread, mean)
        s["gamma"], s["beta"] = 1.0 + 0.2 * randn(c), 0.2 * randn(c)
        if case["grad"]:
            s["dy"] = maps(0.1, 0.01)
    elif case["op"] == "class_loss":
        rows, f, v = case["rows"], case["features"], case["classes"]
        s["x"] = randn(rows, f).to(torch.bfloat16)
        s["w"] = (randn(v, f) / math.sqrt(f)).to(torch.bfloat16)
        # about one row in sixteen has no label (a target outside the classes)
        t = torch.randint(0, v, (rows,), generator=g, device="cuda", dtype=torch.int32)
        s["target"] = torch.where(torch.rand(rows, generator=g, device="cuda") < 1 / 16, torch.full_like(t, -1), t)
    else:
        rows, ci, co, group, dt = case["rows"], case["c_in"], case["c_out"], case["group"], _DT[case["dtype"]]
        s["x"] = randn(rows, ci).to(dt)
        # codes of a weight quantised to -8..7, stored as 0..15, two a byte, the even channel in the low half
        s["codes"] = torch.randint(0, 256, (co, (ci + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = (0.5 + torch.rand(co, -(-ci // group), generator=g, device="cuda")) / (4.0 * math.sqrt(ci))
        s["scales"] = scale.to(dt)
        s["bias"] = 0.1 * randn(co)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import convolution_nhwc_implicit_gb300 as cl
    if case["op"] == "group_norm":
        n, h, w, c, groups = case["n"], case["h"], case["w"], case["c"], case["groups"]
        s["plan"] = cl.GroupNormPlan(n, h, w, c, groups, dtype=case["dtype"], act=case["act"])
        s["y"] = torch.empty(n, h, w, c, device="cuda", dtype=s["x"].dtype)
        s["mean"], s["rstd"] = (torch.empty(n, groups, device="cuda") for _ in range(2))
        if case["grad"]:
            s["dx"] = torch.empty_like(s["y"])
            s["dgamma"], s["dbeta"] = (torch.empty(c, device="cuda") for _ in range(2))
    elif case["op"] == "class_loss":
        s["plan"] = cl.ClassLossPlan(case["rows"], case["features"], case["classes"])
        s["loss"] = torch.empty((), device="cuda")
        s["lse"] = torch.empty(case["rows"], device="cuda")
        if case["grad"]:
            s["dx"], s["dw"] = (torch.empty(t.shape, device="cuda", dtype=t.dtype) for t in (s["x"], s["w"]))
    else:
        s["plan"] = cl.W4Plan(case["rows"], case["c_in"], case["c_out"], group=case["group"], dtype=case["dtype"],
                              act=case["act"])
        s["packed"] = s["plan"].pack(s["codes"])  # laid out once, as a program that serves keeps it
        s["y"] = torch.empty(case["rows"], case["c_out"], device="cuda", dtype=s["x"].dtype)
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"group_norm": _own_group_norm, "class_loss": _own_loss, "w4": _own_w4}[op](s)
    return {"group_norm": _plain_group_norm, "class_loss": _plain_loss, "w4": _plain_w4}[op](s)


def _own_group_norm(s):
    p = s["plan"]
    p.run(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"])
    out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if s["case"]["grad"]:
        p.run_backward(s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], s["dy"], s["dx"], s["dgamma"], s["dbeta"])
        out.update(dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    return out


def _own_loss(s):
    p = s["plan"]
    p.run(s["x"], s["w"], s["target"], s["loss"], s["lse"])
    out = {"loss": s["loss"], "lse": s["lse"]}
    if s["case"]["grad"]:
        p.run_backward(s["x"], s["w"], s["target"], s["lse"], s["dx"], s["dw"])
        out.update(dx=s["dx"], dw=s["dw"])
    return out


def _own_w4(s):
    s["plan"].run(s["x"], s["packed"], s["scales"], s["bias"], s["y"])
    return s["y"]


def _plain_group_norm(s):
    case, dt = s["case"], s["x"].dtype
    n, h, w, c, groups = case["n"], case["h"], case["w"], case["c"], case["groups"]
    shape = (n, h * w, groups, c // groups)
    gamma, beta = s["gamma"].view(1, 1, groups, -1), s["beta"].view(1, 1, groups, -1)
    x = s["x"].float().reshape(shape)
    mean = x.mean(dim=(1, 3), keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=(1, 3), keepdim=True) + 1e-5)
    xhat = xc * rstd
    z = xhat * gamma + beta
    if case["act"] == "mish":
        t = torch.tanh(torch.log1p(torch.exp(z)))
        y = z * t
    elif case["act"] == "relu":
        y = torch.clamp(z, min=0.0)
    else:
        y = z
    out = {"y": y.reshape(n, h, w, c).to(dt), "mean": mean.reshape(n, groups), "rstd": rstd.reshape(n, groups)}
    if case["grad"]:
        dz = s["dy"].float().reshape(shape)
        if case["act"] == "mish":
            dz = dz * (t + z * (1.0 - t * t) / (1.0 + torch.exp(-z)))
        elif case["act"] == "relu":
            dz = dz * (z > 0)
        out["dgamma"] = (dz * xhat).sum(dim=(0, 1)).reshape(c)
        out["dbeta"] = dz.sum(dim=(0, 1)).reshape(c)
        dxhat = dz * gamma
        dx = rstd * (dxhat - dxhat.mean(dim=(1, 3), keepdim=True) - xhat * (dxhat * xhat).mean(dim=(1, 3), keepdim=True))
        out["dx"] = dx.reshape(n, h, w, c).to(dt)
    return out


def _plain_loss(s):
    x, w, target = s["x"].float(), s["w"].float(), s["target"].long()
    logits = x @ w.t()
    top = logits.max(dim=1, keepdim=True).values
    lse = (top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True)))
    here = (target >= 0) & (target < w.shape[0])
    at = torch.where(here, target, torch.zeros_like(target)).unsqueeze(1)
    each = torch.where(here, lse.squeeze(1) - logits.gather(1, at).squeeze(1), torch.zeros_like(lse.squeeze(1)))
    count = here.sum().clamp(min=1).float()
    out = {"loss": each.sum() / count, "lse": lse.squeeze(1)}
    if s["case"]["grad"]:
        g = torch.exp(logits - lse)
        g = g.scatter_add(1, at, -torch.ones_like(lse))
        g = g * (here.float() / count).unsqueeze(1)
        out["dx"] = (g @ w).to(s["x"].dtype)
        out["dw"] = (g.t() @ x).to(s["w"].dtype)
    return out


def _plain_w4(s):
    case = s["case"]
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=2).flatten(1)[:, :case["c_in"]]
    scale = s["scales"].float().repeat_interleave(case["group"], dim=1)[:, :case["c_in"]]
    y = s["x"].float() @ ((codes.float() - 8.0) * scale).t() + s["bias"]
    if case["act"] == "mish":
        y = y * torch.tanh(torch.log1p(torch.exp(y)))
    elif case["act"] == "relu":
        y = torch.clamp(y, min=0.0)
    return y.to(s["x"].dtype)


# ----------------------------------------------------------------------- work
def work(case):
    if case["op"] == "group_norm":
        m = case["n"] * case["h"] * case["w"] * case["c"]
        small = 8 * case["c"] + 8 * case["n"] * case["groups"]
        moves, flops = (4, 30) if case["grad"] else (2, 10)
        return {"bytes": m * _ES[case["dtype"]] * moves + small, "flops": m * flops}
    if case["op"] == "class_loss":
        n, f, v = case["rows"], case["features"], case["classes"]
        times = 2 if case["grad"] else 1
        return {"bytes": 2 * f * (n + v) * times + 8 * n, "flops": 2 * n * f * v * (3 if case["grad"] else 1)}
    n, ci, co = case["rows"], case["c_in"], case["c_out"]
    es = _ES[case["dtype"]]
    return {"bytes": co * ((ci + 1) // 2) + co * -(-ci // case["group"]) * es + n * (ci + co) * es + 4 * co,
            "flops": 2 * n * ci * co}


# ---------------------------------------------------------- the 64-bit answers
def exact(case, seed):
    s = _inputs(case, seed)
    return {"group_norm": _exact_group_norm, "class_loss": _exact_loss, "w4": _exact_w4}[case["op"]](case, s)


def _exact_act(z, act):
    """act(z) and its derivative, in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    # tanh(log(1 + e)) = q / (q + 2), q = e^2 + 2 e; its derivative by z: 4 e (1 + e) / (q + 2)^2
    e = torch.exp(z.clamp(max=40.0))
    q = e * (e + 2)
    t = q / (q + 2)
    return z * t, t + z * 4 * e * (1 + e) / (q + 2) ** 2


def _exact_group_norm(case, s):
    n, c, groups = case["n"], case["c"], case["groups"]
    y, mean, rstd, dx = [], [], [], []
    dgamma, dbeta = torch.zeros(c, device="cuda", dtype=torch.float64), torch.zeros(c, device="cuda", dtype=torch.float64)
    gamma, beta = s["gamma"].double(), s["beta"].double()
    for i in range(n):  # one image at a time, its groups as rows
        x = s["x"][i].reshape(-1, groups, c // groups).transpose(0, 1).reshape(groups, -1).double()
        var, mu = torch.var_mean(x, dim=1, unbiased=False)
        r = (var + 1e-5).rsqrt()

        def back(v):
            return v.reshape(groups, -1, c // groups).transpose(0, 1).reshape(case["h"], case["w"], c)

        xhat = back((x - mu[:, None]) * r[:, None])
        z, dact = _exact_act(xhat * gamma + beta, case["act"])
        y.append(z)
        mean.append(mu)
        rstd.append(r)
        if case["grad"]:
            dz = s["dy"][i].double() * dact
            dgamma += (dz * xhat).sum(dim=(0, 1))
            dbeta += dz.sum(dim=(0, 1))
            gh = (dz * gamma).reshape(-1, groups, c // groups)
            xg = xhat.reshape(-1, groups, c // groups)
            m = gh.shape[0] * gh.shape[2]
            a, b = gh.sum(dim=(0, 2)) / m, (gh * xg).sum(dim=(0, 2)) / m
            d = r[:, None] * (gh - a[:, None] - xg * b[:, None])
            dx.append(d.reshape(case["h"], case["w"], c))
    out = {"y": torch.stack(y), "mean": torch.stack(mean), "rstd": torch.stack(rstd)}
    if case["grad"]:
        out.update(dx=torch.stack(dx), dgamma=dgamma, dbeta=dbeta)
    return out


def _exact_loss(case, s):
    rows, v = case["rows"], case["classes"]
    w = s["w"].double()
    ok = (s["target"] >= 0) & (s["target"] < v)
    count = max(1, int(ok.sum()))
    total, lse, dx = 0.0, [], []
    dw = torch.zeros_like(w) if case["grad"] else None
    step = max(1, (1 << 26) // v)
    for i in range(0, rows, step):
        x = s["x"][i:i + step].double()
        z = x @ w.t()
        l = torch.logsumexp(z, dim=1)
        lse.append(l)
        r = ok[i:i + step].nonzero().squeeze(1)
        t = s["target"][i:i + step].long()[r]
        total += float((l[r] - z[r, t]).sum())
        if case["grad"]:
            p = torch.softmax(z, dim=1)
            p[r, t] -= 1.0
            p *= ok[i:i + step, None].double() / count
            dx.append(p @ w)
            dw += p.t() @ x
    out = {"loss": torch.tensor(total / count, dtype=torch.float64), "lse": torch.cat(lse)}
    if case["grad"]:
        out.update(dx=torch.cat(dx), dw=dw)
    return out


def _exact_w4(case, s):
    ci = case["c_in"]
    x = s["x"].double()
    y = []
    for i in range(0, case["c_out"], 4096):
        b = s["codes"][i:i + 4096].to(torch.int64)
        q = torch.empty(b.shape[0], 2 * b.shape[1], device=b.device, dtype=torch.float64)
        q[:, 0::2], q[:, 1::2] = (b % 16).double(), (b // 16).double()
        group = torch.arange(ci, device=b.device) // case["group"]
        y.append(x @ ((q[:, :ci] - 8) * s["scales"][i:i + 4096].double()[:, group]).t())
    z = torch.cat(y, dim=1) + s["bias"].double()
    return _exact_act(z, case["act"])[0]
