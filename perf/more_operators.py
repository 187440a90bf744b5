"""What is measured of two more operators around the convolution layers: the
norms before and after a block, fused with the block's gate, its residual scale
and the residual add (channels last, forward and gradient), and the global norm
of many gradients with clipping.

Each case runs in two forms that take the same inputs: a plain one in
elementary torch operations and 32 bits (64 for the sum over all gradients),
rounded once at the end, and, where ``own`` is true, this package's entry
points.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_EPS = 1e-5
_MOST_MAP = 8192 * 8192                  # elements of the largest map, forward
_MOST_MAP_GRAD = 16 * 160 * 160 * 128    # ... and in training
_MOST_GRADS = 9 * 24 * 2048 * 2048       # elements of the largest set of gradients, about


# ------------------------------------------------------------------ the cases
def _norm(name, n, h, w, c, post, pre, dtype, grad, gate, wide=0):
    return {"name": name, "op": "block_norm", "n": n, "h": h, "w": w, "c": c, "post": post, "pre": pre, "dtype": dtype,
            "grad": grad, "gate": gate, "wide": wide}


def _clip(name, blocks, width, classes, max_norm, in_place, flat):
    return {"name": name, "op": "grad_clip", "blocks": blocks, "width": width, "classes": classes,
            "max_norm": max_norm, "in_place": in_place, "flat": flat}


def listed():
    return [
        # one pooled feature vector between two blocks: only latency counts
        _norm("norm_1x512_bf16", 1, 1, 1, 512, "none", "layer", "bf16", False, False),
        # after the batch-8 3x3 256->256 layer of the throughput sweep, both norms and a gate for each image
        _norm("norm_80x80x256_b8_bf16", 8, 80, 80, 256, "rms", "rms", "bf16", False, True),
        # an odd number of channels, keyword-spotting sized maps, fp32
        _norm("norm_25x5x61_b64_f32", 64, 25, 5, 61, "layer", "layer", "f32", False, False),
        # long rows: a prompt through a wide block
        _norm("norm_8192x8192_bf16", 1, 1, 8192, 8192, "rms", "rms", "bf16", False, False),
        # the last stage of a small classifier in training, two images
        _norm("norm_grad_7x7x512_b2_bf16", 2, 7, 7, 512, "layer", "layer", "bf16", True, True),
        # the sweep's pointwise layer's maps in training, a gate for each image
        _norm("norm_grad_20x20x1024_b8_bf16", 8, 20, 20, 1024, "none", "rms", "bf16", True, True),
        # channel slices of concatenated buffers, groups of channels that fill no 16 bytes
        _norm("norm_grad_slice_40x40x510_b8_bf16", 8, 40, 40, 510, "layer", "rms", "bf16", True, False, 510),
        # a training batch in fp32, larger than the L2
        _norm("norm_grad_160x160x128_b16_f32", 16, 160, 160, 128, "rms", "layer", "f32", True, False),
        # a class head with a norm or two below it: only latency counts
        _clip("clip_1_128_1000", 1, 128, 1000, 1.0, False, False),
        # a small network's gradients as views of flat buffers, at odd addresses
        _clip("clip_12_509_10007_flat", 12, 509, 10007, 1.0, False, True),
        # gradients that need no clipping, in place: one read
        _clip("clip_16_1024_32003_under", 16, 1024, 32003, 1.0e6, True, False),
        # a billion gradients
        _clip("clip_24_2048_50000", 24, 2048, 50000, 1.0, False, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.65:
        grad = rng.random() < 0.5
        while True:
            c = _log(rng, 8, 8192)
            if rng.random() < 0.7:
                c = -(-c // 8) * 8
            n, h, w = _log(rng, 1, 64), _log(rng, 1, 160), _log(rng, 1, 160)
            dtype = rng.choice(["bf16", "bf16", "f32"])
            wide = rng.choice([0, 0, c])
            most = _MOST_MAP_GRAD if grad else _MOST_MAP if dtype == "bf16" else _MOST_MAP // 2
            if n * h * w * c <= most:
                break
        post = rng.choice(["none", "layer", "rms"])
        case = _norm("", n, h, w, c, post, rng.choice(["layer", "rms"]), dtype, grad, rng.random() < 0.5, wide)
    else:
        while True:
            blocks, width, classes = _log(rng, 1, 48), _log(rng, 16, 2048), _log(rng, 10, 50000)
            if 9 * blocks * width * width + classes * width <= _MOST_GRADS:
                break
        under = rng.random() < 0.3
        case = _clip("", blocks, width, classes, 1.0e6 if under else rng.choice([0.01, 0.1, 1.0]), under,
                     rng.random() < 0.4)
    del case["name"]
    return case


def _grad_sizes(case):
    """Elements and type of each gradient: blocks of three matrices and four
    vectors, then a class head."""
    c = case["width"]
    one = [(c * c, "bf16"), (4 * c * c, "bf16"), (4 * c * c, "bf16"), (c, "f32"), (c, "f32"), (c, "f32"), (4 * c, "f32")]
    return one * case["blocks"] + [(case["classes"] * c, "bf16")]


# ----------------------------------------------------------------- the inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _places(case):
    """Where each gradient lies: its type, first element and elements, in one
    buffer for each type; and the buffers' elements.  Each starts at a multiple
    of 256, or, flat, where the one before it ends, the first at element 1."""
    ends = {d: 1 if case["flat"] else 0 for d in _DT}
    places = []
    for k, d in _grad_sizes(case):
        at = ends[d] if case["flat"] else -(-ends[d] // 256) * 256
        places.append((d, at, k))
        ends[d] = at + k
    return places, ends


def _buffers(case):
    """Zeroed memory of every gradient: the buffers and the gradients in them."""
    places, ends = _places(case)
    flat = {d: torch.zeros(k, device="cuda", dtype=_DT[d]) for d, k in ends.items()}
    return flat, [flat[d][at:at + k] for d, at, k in places]


def _inputs(case, seed):
    g = _generator(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s = {}
    if case["op"] == "block_norm":
        n, h, w, c, dt = case["n"], case["h"], case["w"], case["c"], _DT[case["dtype"]]

        def maps(scale, shift):
            buf = torch.empty(n, h, w, c + case["wide"], device="cuda", dtype=dt)
            view = buf[..., case["wide"]:]
            view.copy_(randn(n, h, w, c) * scale + shift)
            return view

        # a residual stream whose channels have means of their own, and a block's output of another size
        s["x"] = maps(0.5 + torch.rand(c, generator=g, device="cuda"), 0.5 * randn(c))
        s["f"] = maps(2.0 * (0.5 + torch.rand(c, generator=g, device="cuda")), 0.3 * randn(c))
        s["scale"] = 0.3 + 0.1 * randn(c)
        s["gate"] = torch.sigmoid(randn(n, c)) if case["gate"] else None
        for k in ("post", "pre"):
            kind = case[k]
            s[k + "_gamma"] = None if kind == "none" else 1.0 + 0.2 * randn(c)
            s[k + "_beta"] = 0.2 * randn(c) if kind == "layer" else None
        if case["grad"]:
            s["dy"], s["dz"] = maps(0.1, 0.01), maps(0.1, 0.01)
    else:
        s["flat"], s["grads"] = _buffers(case)
        for t in s["grads"]:  # matrices' gradients are smaller than vectors'
            t.copy_((0.01 if t.dtype is torch.bfloat16 else 0.05) * randn(t.numel()))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import convolution_nhwc_implicit_gb300 as cl
    if case["op"] == "block_norm":
        n, h, w, c = case["n"], case["h"], case["w"], case["c"]
        s["plan"] = cl.BlockNormPlan(n, h, w, c, post=case["post"], pre=case["pre"], eps=_EPS, dtype=case["dtype"])
        s["y"], s["z"] = (torch.empty(n, h, w, c, device="cuda", dtype=s["x"].dtype) for _ in range(2))
        s["stats"] = torch.empty(n, h, w, 4, device="cuda")
        if case["grad"]:
            s["dx"], s["df"] = (torch.empty_like(s["y"]) for _ in range(2))
            for k in ("scale", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta"):
                s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
    else:
        s["plan"] = cl.GradClipPlan([t.shape for t in s["grads"]], [d for _, d in _grad_sizes(case)])
        s["norm"] = torch.empty((), device="cuda")
        s["flat_out"], s["out"] = (s["flat"], None) if case["in_place"] else _buffers(case)
    return s


# ------------------------------------------------------------------- one pass
def run(s):
    norm = s["case"]["op"] == "block_norm"
    if own:
        return _own_block_norm(s) if norm else _own_grad_clip(s)
    return _plain_block_norm(s) if norm else _plain_grad_clip(s)


_GRADS = ("dscale", "dgate", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")


def _own_block_norm(s):
    p = s["plan"]
    p.run(s["x"], s["f"], s["y"], s["z"], s["stats"], scale=s["scale"], gate=s["gate"], post_gamma=s["post_gamma"],
          post_beta=s["post_beta"], pre_gamma=s["pre_gamma"], pre_beta=s["pre_beta"])
    out = {"y": s["y"], "z": s["z"], "stats": s["stats"]}
    if s["case"]["grad"]:
        p.run_backward(s["x"], s["f"], s["stats"], s["dy"], s["dz"], s["dx"], s["df"], scale=s["scale"], gate=s["gate"],
                       post_gamma=s["post_gamma"], post_beta=s["post_beta"], pre_gamma=s["pre_gamma"],
                       dscale=s["dscale"], dgate=s["dgate"], dpost_gamma=s["dpost_gamma"], dpost_beta=s["dpost_beta"],
                       dpre_gamma=s["dpre_gamma"], dpre_beta=s["dpre_beta"])
        out.update(dx=s["dx"], df=s["df"])
        out.update((k, s[k]) for k in _GRADS if s[k] is not None)
    return out


def _own_grad_clip(s):
    s["plan"].run(s["grads"], s["case"]["max_norm"], s["norm"], out=s["out"])
    return {"norm": s["norm"], "grads": s["flat_out"]}


def _plain_statistics(v, kind):
    mean = v.mean(dim=-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    if kind == "none":
        return mean, torch.ones_like(mean)
    d = v - mean
    return mean, 1.0 / torch.sqrt((d * d).mean(dim=-1, keepdim=True) + _EPS)


def _plain_affine(v, gamma, beta):
    v = v if gamma is None else v * gamma
    return v if beta is None else v + beta


def _plain_through_norm(d, hat, rstd, kind):
    """The gradient at a norm's input from that at its normalised values."""
    if kind == "none":
        return d
    d = d - hat * (d * hat).mean(dim=-1, keepdim=True) - (d.mean(dim=-1, keepdim=True) if kind == "layer" else 0.0)
    return d * rstd


def _plain_block_norm(s):
    case, dt = s["case"], s["x"].dtype
    post, pre = case["post"], case["pre"]
    x, f = s["x"].float(), s["f"].float()
    m1, r1 = _plain_statistics(f, post)
    uhat = (f - m1) * r1
    u = _plain_affine(uhat, s["post_gamma"], s["post_beta"])
    factor = s["scale"] if s["gate"] is None else (s["scale"] * s["gate"])[:, None, None, :]
    y = x + factor * u
    m2, r2 = _plain_statistics(y, pre)
    yhat = (y - m2) * r2
    z = _plain_affine(yhat, s["pre_gamma"], s["pre_beta"])
    out = {"y": y.to(dt), "z": z.to(dt), "stats": torch.cat([m1, r1, m2, r2], dim=-1)}
    if case["grad"]:
        dz = s["dz"].float()
        dyy = s["dy"].float() + _plain_through_norm(_plain_affine(dz, s["pre_gamma"], None), yhat, r2, pre)
        du = factor * dyy
        df = _plain_through_norm(_plain_affine(du, s["post_gamma"], None), uhat, r1, post)
        out.update(dx=dyy.to(dt), df=df.to(dt))
        per_image = (dyy * u).sum(dim=(1, 2))
        out["dscale"] = (per_image if s["gate"] is None else per_image * s["gate"]).sum(dim=0)
        if s["gate"] is not None:
            out["dgate"] = per_image * s["scale"]
        if s["post_gamma"] is not None:
            out["dpost_gamma"] = (du * uhat).sum(dim=(0, 1, 2))
        if s["post_beta"] is not None:
            out["dpost_beta"] = du.sum(dim=(0, 1, 2))
        out["dpre_gamma"] = (dz * yhat).sum(dim=(0, 1, 2))
        if s["pre_beta"] is not None:
            out["dpre_beta"] = dz.sum(dim=(0, 1, 2))
    return out


def _plain_grad_clip(s):
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for g in s["grads"]:
        v = g.float()
        total = total + (v * v).sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    factor = torch.clamp(s["case"]["max_norm"] / (norm + 1e-6), max=1.0)
    flat, out = _buffers(s["case"])
    for g, o in zip(s["grads"], out):
        o.copy_(g.float() * factor)
    return {"norm": norm, "grads": flat}


# ----------------------------------------------------------------------- work
def work(case):
    if case["op"] == "block_norm":
        rows, c = case["n"] * case["h"] * case["w"], case["c"]
        m = rows * c
        vectors = 1 + case["n"] * case["gate"] + sum({"none": 0, "rms": 1, "layer": 2}[case[k]] for k in ("post", "pre"))
        maps, flops, small = 4, 20, 16 * rows + 4 * c * vectors
        if case["grad"]:
            maps, flops, small = 10, 65, 2 * 16 * rows + 3 * 4 * c * vectors
        return {"bytes": maps * m * _ES[case["dtype"]] + small, "flops": flops * m}
    sizes = _grad_sizes(case)
    total = sum(k * _ES[d] for k, d in sizes)
    written = 0 if case["in_place"] else total
    count = sum(k for k, _ in sizes)
    return {"bytes": total + written + 4, "flops": (2 if case["in_place"] else 3) * count}


# ---------------------------------------------------------- the 64-bit answers
def exact(case, seed):
    s = _inputs(case, seed)
    return _exact_block_norm(case, s) if case["op"] == "block_norm" else _exact_grad_clip(case, s)


def _exact_norm(rows, kind):
    """Normalised rows, their means and their reciprocal deviations, in 64 bits."""
    zero = torch.zeros(rows.shape[0], device=rows.device, dtype=torch.float64)
    if kind == "none":
        return rows, zero, zero + 1
    if kind == "rms":
        r = (rows.square().sum(1) / rows.shape[1] + _EPS).rsqrt()
        return rows * r[:, None], zero, r
    var, mu = torch.var_mean(rows, dim=1, unbiased=False)
    r = (var + _EPS).rsqrt()
    return (rows - mu[:, None]) * r[:, None], mu, r


def _exact_back(d, hat, r, kind):
    if kind == "none":
        return d
    along = torch.einsum("rc,rc->r", d, hat) / d.shape[1]
    d = torch.addcmul(d, hat, along[:, None], value=-1.0)
    if kind == "layer":
        d = d - d.mean(1, keepdim=True)
    return d * r[:, None]


def _exact_block_norm(case, s):
    n, h, w, c = case["n"], case["h"], case["w"], case["c"]
    one = torch.ones(c, device="cuda", dtype=torch.float64)
    vec = {k: None if s[k] is None else s[k].double() for k in ("scale", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta")}
    g1, g2 = (one if vec[k] is None else vec[k] for k in ("post_gamma", "pre_gamma"))
    b1, b2 = (0 * one if vec[k] is None else vec[k] for k in ("post_beta", "pre_beta"))
    y, z, stats = (torch.empty(n, h * w, k, device="cuda", dtype=torch.float64) for k in (c, c, 4))
    if case["grad"]:
        dx, df = torch.empty_like(y), torch.empty_like(y)
        sums = {k: None if vec[k] is None else torch.zeros_like(vec[k]) for k in vec}
    step = max(1, (1 << 24) // c)
    for i in range(n):  # one image at a time, its pixels as rows
        gate = one if vec["gate"] is None else vec["gate"][i]
        for a in range(0, h * w, step):
            def rows(k):
                return s[k][i].reshape(h * w, c)[a:a + step].double()
            at = slice(a, min(a + step, h * w))
            fh, m1, r1 = _exact_norm(rows("f"), case["post"])
            u = fh * g1 + b1
            yy = rows("x") + u * (vec["scale"] * gate)
            yh, m2, r2 = _exact_norm(yy, case["pre"])
            y[i, at], z[i, at] = yy, yh * g2 + b2
            stats[i, at] = torch.stack([m1, r1, m2, r2], dim=1)
            if case["grad"]:
                dz = rows("dz")
                t = rows("dy") + _exact_back(dz * g2, yh, r2, case["pre"])
                v = t * (vec["scale"] * gate)
                dx[i, at], df[i, at] = t, _exact_back(v * g1, fh, r1, case["post"])
                tu = (t * u).sum(0)
                sums["scale"] += tu * gate
                if vec["gate"] is not None:
                    sums["gate"][i] += tu * vec["scale"]
                for k, term in (("post_gamma", (v * fh).sum(0)), ("post_beta", v.sum(0)), ("pre_gamma", (dz * yh).sum(0)),
                                ("pre_beta", dz.sum(0))):
                    if sums[k] is not None:
                        sums[k] += term
    out = {"y": y.view(n, h, w, c), "z": z.view(n, h, w, c), "stats": stats.view(n, h, w, 4)}
    if case["grad"]:
        out.update(dx=dx.view(n, h, w, c), df=df.view(n, h, w, c))
        out.update(("d" + k, v) for k, v in sums.items() if v is not None)
    return out


def _exact_grad_clip(case, s):
    step = 1 << 26
    pieces = [float(torch.linalg.vector_norm(g[i:i + step], dtype=torch.float64)) for g in s["grads"]
              for i in range(0, g.numel(), step)]
    norm = math.sqrt(math.fsum(v * v for v in pieces))
    factor = min(1.0, case["max_norm"] / (norm + 1e-6))
    # (what lies between the gradients is zero)
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": {d: t.double() * factor for d, t in s["flat"].items()}}
