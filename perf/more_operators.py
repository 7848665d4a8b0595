"""Rotary positions of attention heads, norms of queries and keys with the
rotation in the same pass, and dropout from a counter-based generator: the
cases they are timed on, their plain forms in 32 bits and their definitions in
64 bits.

A case is one call (serving) or one forward and backward pass (training) of an
operator.  ``run`` computes it by elementary tensor operations, or, with
``own`` set, by the calls of ``sparse_convolution_gb300``.
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0
SLOW, FAST = 1.0, 32.0  # turns over the trained length between which a channel is partly stretched
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    def heads(name, op, n, heads, kv_heads, d, rot, axes, layout, dtype, span, scaling="none", factor=1.0, length=0,
              fused=False, pad=0):
        return {"name": name, "op": op, "n": n, "heads": heads, "kv_heads": kv_heads, "d": d, "rot": rot, "axes": axes,
                "layout": layout, "dtype": dtype, "span": span, "scaling": scaling, "factor": factor, "length": length,
                "fused": fused, "pad": pad}

    return [
        # one new token far into a stretched context, shared key heads: serving, latency
        heads("rotate_one_token", "rotate", 1, 16, 4, 128, 128, 1, "half", "bf16", 1 << 17, "parts", 8.0, 8192),
        # a prompt in fp32, an odd length, 60 of 100 channels rotated, heads inside wider rows
        heads("rotate_prompt_odd", "rotate", 4099, 8, 8, 100, 60, 1, "interleaved", "f32", 1 << 15, "linear", 4.0, 0,
              False, 3),
        # a lidar frame's voxels by their three coordinates, a training step
        heads("rotate_train_voxels", "rotate_train", 150001, 8, 8, 64, 64, 3, "half", "bf16", 1440),
        # one new token whose queries and keys lie in one product's row: serving, latency
        heads("norm_rotate_one_token", "norm_rotate", 1, 16, 4, 128, 64, 1, "interleaved", "bf16", 1 << 17, "base", 4.0, 0,
              True),
        # a lidar frame's voxels in serving, wide heads, shared key heads, out of one product's rows
        heads("norm_rotate_voxels", "norm_rotate", 150001, 8, 2, 128, 128, 3, "half", "bf16", 1440, fused=True),
        # an ordinary training step: ragged samples' tokens end to end, shared key heads
        heads("norm_rotate_train", "norm_rotate_train", 9014, 8, 2, 64, 64, 1, "half", "bf16", 4003, fused=True),
        # a small fp32 model's training step: odd head size, part of the head rotated by two coordinates
        heads("norm_rotate_train_odd", "norm_rotate_train", 30011, 6, 3, 40, 28, 2, "interleaved", "f32", 1024),
        # every voxel of a large grid, the widest training step
        heads("norm_rotate_train_large", "norm_rotate_train", 1000000, 8, 8, 64, 64, 3, "half", "bf16", 2048),
        # one voxel's features added to its stream: latency
        {"name": "dropout_one_row", "op": "dropout", "n": 1, "c": 256, "dtype": "bf16", "p": 0.1, "residual": True,
         "pad": 0},
        # a single scan's voxels in fp32, an odd channel count, rows inside a wider tensor
        {"name": "dropout_train_odd", "op": "dropout_train", "n": 30011, "c": 101, "dtype": "f32", "p": 0.25,
         "residual": False, "pad": 33},
        # a lidar frame's block of 256 channels added to its stream
        {"name": "dropout_train_lidar", "op": "dropout_train", "n": 150001, "c": 256, "dtype": "bf16", "p": 0.1,
         "residual": True, "pad": 0},
        # the batched narrow band's 32-channel activations
        {"name": "dropout_train_large", "op": "dropout_train", "n": 10000000, "c": 32, "dtype": "bf16", "p": 0.1,
         "residual": True, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_train", "norm_rotate", "norm_rotate", "norm_rotate_train", "norm_rotate_train",
                     "dropout", "dropout_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("dropout"):
        c = _log_int(rng, 8, 1024)
        if rng.random() < 0.5:
            c = max(8, c // 8 * 8)
        n = _log_int(rng, 1, (200_000_000 if dtype == "bf16" else 100_000_000) // c)
        return {"op": op, "n": n, "c": c, "dtype": dtype, "p": rng.choice([0.0, 0.05, 0.1, 0.25, 0.5, 0.9]),
                "residual": rng.random() < 0.5, "pad": rng.choice([0, 0, 8, 33])}
    kv_heads, shared = rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4, 8])
    d = rng.choice([16, 32, 40, 64, 64, 80, 96, 100, 128, 128, 192, 256])
    heads = kv_heads * shared
    n = _log_int(rng, 1, (800_000_000 if dtype == "bf16" else 400_000_000) // ((heads + kv_heads) * d))
    axes = rng.choice([1, 1, 2, 3])
    rot = d if rng.random() < 0.6 else max(2 * axes, 2 * rng.randint(1, d // 2))
    scaling = rng.choice(["none", "none", "linear", "base", "parts"]) if axes == 1 else "none"
    return {"op": op, "n": n, "heads": heads, "kv_heads": kv_heads, "d": d, "rot": rot, "axes": axes,
            "layout": rng.choice(["half", "interleaved"]), "dtype": dtype,
            "span": _log_int(rng, 128, 1 << 20) if axes == 1 else _log_int(rng, 64, 4096), "scaling": scaling,
            "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 16.0]),
            "length": 8192 if scaling == "parts" else 0, "fused": rng.random() < 0.4, "pad": rng.choice([0, 0, 0, 1, 8])}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, n, pad = DTYPES[case["dtype"]], case["n"], case["pad"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def rows(*shape, out=None, spread=1.0):
        # of the case's type, a part at a time: the fp32 values would be twice as large
        out = torch.empty(*shape, device="cuda", dtype=dtype) if out is None else out
        step = max(1, (1 << 27) // max(1, math.prod(shape[1:])))
        for i in range(0, shape[0], step):
            out[i:i + step] = (normal(min(step, shape[0] - i), *shape[1:]) * spread).to(dtype)
        return out

    if case["op"].startswith("dropout"):
        c = case["c"]
        x = torch.empty(n, c + pad, device="cuda", dtype=dtype)
        x[:, c:] = 0
        state = {"case": dict(case), "x": rows(n, c, out=x[:, :c]), "residual": None,
                 "seed": (seed * 1000003 + 12345) % (1 << 40), "offset": seed % 1000}
        if case["residual"]:
            state["residual"] = rows(n, c, spread=2.0)
        if case["op"].endswith("train"):
            state["dy"] = rows(n, c)
        return state

    h, hk, d, axes = case["heads"], case["kv_heads"], case["d"], case["axes"]
    # a product's outputs: channels of different spread
    if case["fused"]:  # queries, keys and values of a token in one row
        qkv = torch.empty(n, h + 2 * hk, d + pad, device="cuda", dtype=dtype)
        qkv[:, :, d:] = 0
        qkv[:, h + hk:] = 0
        q, k = qkv[:, :h, :d], qkv[:, h:h + hk, :d]
    else:
        q, k = (torch.empty(n, m, d + pad, device="cuda", dtype=dtype) for m in (h, hk))
        q[:, :, d:] = 0
        k[:, :, d:] = 0
        q, k = q[:, :, :d], k[:, :, :d]
    spread = torch.exp(0.5 * normal(d))
    rows(n, h, d, out=q, spread=spread)
    rows(n, hk, d, out=k, spread=spread)
    if axes == 1:  # token positions, samples end to end: runs that start anywhere
        start = torch.randint(0, case["span"], (-(-n // 997),), device="cuda", generator=g)
        at = (start[:, None] + torch.arange(997, device="cuda")).reshape(-1)[:n] % case["span"]
    else:  # voxel coordinates
        at = torch.randint(-case["span"], case["span"], (n, axes), device="cuda", generator=g)
    state = {"case": dict(case), "q": q, "k": k, "positions": at.to(torch.int32)}
    if own:
        import sparse_convolution_gb300 as fvx

        state["rotary"] = fvx.Rotary(case["rot"], axes=axes, base=BASE, layout=case["layout"],
                                     scaling=None if case["scaling"] == "none" else case["scaling"],
                                     factor=case["factor"], length=case["length"] or None)
    if case["op"].startswith("norm"):
        state["wq"], state["wk"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
    if case["op"].endswith("train"):
        state["dq"], state["dk"] = rows(n, h, d), rows(n, hk, d)
    return state


# ---------------------------------------------------------------- plain forms
def _frequencies(case):
    """Radians per step of every rotated pair (64 bits), its axis, and the factor on the rotated values."""
    pairs, axes = case["rot"] // 2, case["axes"]
    out, axis = [], []
    for a in range(axes):
        own_pairs = pairs // axes + (a < pairs % axes)
        base = BASE
        if case["scaling"] == "base" and own_pairs > 1:
            base *= case["factor"] ** (own_pairs / (own_pairs - 1))
        f = torch.tensor([base ** (-i / own_pairs) for i in range(own_pairs)], dtype=torch.float64)
        if case["scaling"] == "linear":
            f = f / case["factor"]
        if case["scaling"] == "parts":
            keep = ((case["length"] * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
            f = f * (keep + (1 - keep) / case["factor"])
        out.append(f)
        axis += [a] * own_pairs
    size = 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "parts" else 1.0
    return torch.cat(out).cuda(), axis, size


def _angles(s):
    f, axis, size = _frequencies(s["case"])
    at = s["positions"].view(s["positions"].shape[0], -1)[:, axis]
    turn = at.double() * f  # far positions: 32 bits would lose the angle
    return (torch.cos(turn) * size).float()[:, None], (torch.sin(turn) * size).float()[:, None]


def _turn(x, cos, sin, case):
    rot, half = case["rot"], case["layout"] == "half"
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if half else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _unit(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _philox(first, count, seed, offset):
    """128 random bits for each of `count` counters from `first` on, as four int64 tensors of 32 bits (Philox 4x32-10,
    Salmon et al. 2011)."""
    low = 0xFFFFFFFF
    at = torch.arange(first, first + count, device="cuda")
    c = [at & low, at >> 32, torch.full_like(at, offset & low), torch.full_like(at, offset >> 32)]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & low) ^ c[1] ^ k0, p1 & low, ((p0 >> 32) & low) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c


def _kept(s):
    """Which values stay: 16 bits each, eight values of the row-major tensor per counter."""
    n, c = s["case"]["n"], s["case"]["c"]
    total, drop = n * c, round(s["case"]["p"] * 65536)
    kept = torch.empty(-(-total // 8), 8, dtype=torch.bool, device="cuda")
    for i in range(0, kept.shape[0], 1 << 24):
        words = _philox(i, min(1 << 24, kept.shape[0] - i), s["seed"], s["offset"])
        for j in range(8):
            kept[i:i + (1 << 24), j] = ((words[j // 2] >> (16 * (j % 2))) & 0xFFFF) >= drop
    return kept.view(-1)[:total].view(n, c), 65536 / (65536 - drop)


def _plain(s):
    case = s["case"]
    op, dtype = case["op"], DTYPES[case["dtype"]]
    if op.startswith("dropout"):
        kept, scale = _kept(s)
        y = torch.where(kept, s["x"].float() * scale, 0)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        if op == "dropout":
            return {"y": y.to(dtype)}
        return {"y": y.to(dtype), "dx": torch.where(kept, s["dy"].float() * scale, 0).to(dtype)}
    cos, sin = _angles(s)
    out = {}
    for name, weight in (("q", "wq"), ("k", "wk")):
        x = s[name].float()
        if op.startswith("rotate"):
            out[name] = _turn(x, cos, sin, case).to(dtype)
            if op.endswith("train"):
                out["d" + name] = _turn(s["d" + name].float(), cos, -sin, case).to(dtype)
            continue
        w, rstd = s[weight], _unit(x)
        out[name] = _turn(x * rstd * w, cos, sin, case).to(dtype)
        if op.endswith("train"):
            g = _turn(s["d" + name].float(), cos, -sin, case)
            unit = x * rstd
            out["d" + weight] = (g * unit).sum((0, 1))
            g = g * w
            out["d" + name] = (rstd * (g - unit * (g * unit).mean(-1, keepdim=True))).to(dtype)
    return out


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import sparse_convolution_gb300 as fvx

    op = s["case"]["op"]
    if op.startswith("dropout"):
        y = fvx.dropout(s["x"], s["case"]["p"], s["seed"], s["offset"], residual=s["residual"])
        if op == "dropout":
            return {"y": y}
        return {"y": y, "dx": fvx.dropout_backward(s["dy"], s["case"]["p"], s["seed"], s["offset"])}
    at, rotary = s["positions"], s["rotary"]
    if op.startswith("rotate"):
        q, k = fvx.rotate_heads(s["q"], at, rotary, k=s["k"])
        if op == "rotate":
            return {"q": q, "k": k}
        dq, dk = fvx.rotate_heads_backward(s["dq"], at, rotary, dk=s["dk"])
        return {"q": q, "dq": dq, "k": k, "dk": dk}
    q, k = fvx.norm_rotate_heads(s["q"], at, rotary, s["wq"], k=s["k"], k_weight=s["wk"], eps=EPS)
    if op == "norm_rotate":
        return {"q": q, "k": k}
    dq, dk, dwq, dwk = fvx.norm_rotate_heads_backward(s["dq"], s["q"], at, rotary, s["wq"], dk=s["dk"], k=s["k"],
                                                      k_weight=s["wk"], eps=EPS)
    return {"q": q, "dwq": dwq, "dq": dq, "k": k, "dwk": dwk, "dk": dk}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the work and the definitions
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    train = case["op"].endswith("train")
    if case["op"].startswith("dropout"):
        e = case["n"] * case["c"]
        return {"bytes": e * size * (2 + case["residual"] + 2 * train), "flops": e * (2 + case["residual"] + train)}
    e = case["n"] * (case["heads"] + case["kv_heads"]) * case["d"]
    turned = e * case["rot"] / case["d"]
    flops = 3 * turned * (1 + train)
    moved = e * size * (4 if train else 2) + 4 * case["n"] * case["axes"]
    if case["op"].startswith("norm"):
        flops += e * (4 + 8 * train)
        moved += 8 * case["d"] * (1 + train)
    return {"bytes": moved, "flops": flops}


def _exact_heads(s):
    case = s["case"]
    rot, d, op = case["rot"], case["d"], case["op"]
    f, axis, size = _frequencies(case)
    places = torch.arange(rot // 2, device="cuda")
    first = places if case["layout"] == "half" else 2 * places
    second = places + rot // 2 if case["layout"] == "half" else 2 * places + 1
    out = {}
    for name in ("q", "k"):
        x_all, heads = s[name], s[name].shape[1]
        w = s["w" + name].double() if op.startswith("norm") else None
        parts, grads, dw = [], [], torch.zeros(d, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // (heads * d))
        for i in range(0, case["n"], step):
            at = s["positions"][i:i + step].view(-1, case["axes"])[:, axis].double()
            spin = torch.polar(torch.full_like(at * f, size), at * f)[:, None]
            x = x_all[i:i + step].double()
            if w is not None:
                norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
                scale = 1 / torch.sqrt(norm ** 2 / d + EPS)
            y = x if w is None else x * scale * w
            pair = torch.complex(y[..., first], y[..., second]) * spin
            y = y.clone()
            y[..., first], y[..., second] = pair.real, pair.imag
            parts.append(y.float() if x_all.numel() > (1 << 24) else y)
            if op.endswith("train"):
                g = s["d" + name][i:i + step].double()
                pair = torch.complex(g[..., first], g[..., second]) * spin.conj()
                g[..., first], g[..., second] = pair.real, pair.imag
                if w is not None:
                    dw += torch.einsum("nhd,nhd->d", g, x * scale)
                    g = g * w * scale - x * (scale ** 3 * ((g * w * x).sum(-1, keepdim=True) / d))
                grads.append(g.float() if x_all.numel() > (1 << 24) else g)
        out[name] = torch.cat(parts)
        if grads:
            out["d" + name] = torch.cat(grads)
            if w is not None:
                out["dw" + name] = dw
    return out


def _exact_kept(first, count, seed, offset, drop):
    """The bits of `count` counters from `first` on; products of 32 bits by halves of 16."""
    def product(x, m):  # the high and the low 32 bits of x * m
        lo, hi = x % 65536, x // 65536
        low = lo * (m % 65536)
        mid = lo * (m // 65536) + hi * (m % 65536) + low // 65536
        return hi * (m // 65536) + mid // 65536, mid % 65536 * 65536 + low % 65536

    i = torch.arange(first, first + count, device="cuda")
    x = torch.stack([i % 2 ** 32, i // 2 ** 32, torch.full_like(i, offset % 2 ** 32), torch.full_like(i, offset // 2 ** 32)])
    for r in range(10):
        key = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        h0, l0 = product(x[0], 0xD2511F53)
        h1, l1 = product(x[2], 0xCD9E8D57)
        x = torch.stack([h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0])
    return torch.stack([x % 65536, x // 65536], 1).reshape(8, count).t().reshape(-1) >= drop


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("dropout"):
        return _exact_heads(s)
    n, c = case["n"], case["c"]
    drop = round(case["p"] * 65536)
    out = {"y": torch.empty(n, c, dtype=torch.float32 if n * c > (1 << 24) else torch.float64, device="cuda")}
    if "dy" in s:
        out["dx"] = torch.empty_like(out["y"])
    step = 8 * max(1, (1 << 21) // c)  # rows of whole counters
    for i in range(0, n, step):
        m = min(step, n - i)
        kept = _exact_kept(i * c // 8, -(-m * c // 8), s["seed"], s["offset"], drop)[:m * c].view(m, c)
        factor = torch.where(kept, 65536 / (65536 - drop), 0.0).double()
        y = s["x"][i:i + m].double() * factor
        out["y"][i:i + m] = y if s["residual"] is None else y + s["residual"][i:i + m].double()
        if "dy" in s:
            out["dx"][i:i + m] = s["dy"][i:i + m].double() * factor
    return out
