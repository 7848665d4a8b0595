"""Layer normalisation of voxel features, activation checkpoints in 8 bits and
cross attention from voxels to an encoder's states: the cases they are timed
on, their plain forms in 32 bits and their definitions in 64 bits.

A case is one call (serving) or one forward and backward pass (training) of an
operator.  ``run`` computes it by elementary tensor operations, or, with
``own`` set, by the calls of ``sparse_convolution_gb300``.
"""
import math

import torch

own = False

EPS = 1e-5
TINY = 2.0 ** -100  # a checkpoint group whose largest magnitude is below this holds zeros
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one voxel's features between two layers of a serving loop: latency
        {"name": "norm_one_row", "op": "norm", "n": 1, "c": 256, "dtype": "bf16", "pad": 0},
        # a single scan's voxels in fp32, an odd channel count, rows inside a wider tensor
        {"name": "norm_train_odd", "op": "norm_train", "n": 30011, "c": 100, "dtype": "f32", "pad": 33},
        # a narrow band at full resolution, the widest tensors of a training step
        {"name": "norm_train_large", "op": "norm_train", "n": 4000000, "c": 64, "dtype": "bf16", "pad": 0},
        # a small grid's activations put away and taken back, channels that end inside a group
        {"name": "pack_small", "op": "pack", "n": 4099, "c": 48, "dtype": "f32", "group": 32, "pad": 0},
        # the batched narrow band's 32-channel activations put away and taken back
        {"name": "pack_large", "op": "pack", "n": 10000000, "c": 32, "dtype": "bf16", "group": 32, "pad": 0},
        # a lidar frame's block of 256 channels trained from 8-bit checkpoints
        {"name": "ck_train_lidar", "op": "ck_train", "n": 150001, "c": 256, "dtype": "bf16", "group": 64, "pad": 0},
        # one query token of each of 8 samples over long encoder states, some of them masked: serving
        {"name": "attend_one_query", "op": "attend", "q_lens": "1,1,1,1,1,1,1,1",
         "kv_lens": "4096,3001,4096,777,2500,4000,1023,4096", "heads": 16, "kv_heads": 4, "d": 128, "drop": 0.2,
         "dtype": "bf16"},
        # voxels of 8 small grids conditioned on short captions: serving
        {"name": "attend_caption", "op": "attend", "q_lens": "4100,3777,5003,1290,4096,3001,812,6007",
         "kv_lens": "77,12,45,77,33,0,64,21", "heads": 8, "kv_heads": 8, "d": 64, "drop": 0.0, "dtype": "bf16"},
        # four large grids over an image encoder's patches, shared key heads
        {"name": "attend_large", "op": "attend", "q_lens": "20000,16384,12345,16807", "kv_lens": "2048,2048,2048,2048",
         "heads": 8, "kv_heads": 4, "d": 128, "drop": 0.0, "dtype": "bf16"},
        # a small fp32 model's training step, odd head size and lengths, an empty sample, masked keys
        {"name": "attend_train_f32", "op": "attend_train", "q_lens": "301,0,777,130", "kv_lens": "50,33,129,7",
         "heads": 6, "kv_heads": 3, "d": 40, "drop": 0.25, "dtype": "f32"},
        # an ordinary training step: ragged samples, shared key heads, masked keys
        {"name": "attend_train_ragged", "op": "attend_train", "q_lens": "1500,2600,911,4003", "kv_lens": "77,1030,333,512",
         "heads": 8, "kv_heads": 2, "d": 64, "drop": 0.1, "dtype": "bf16"},
        # the widest training step: every voxel of two grids over an image encoder's patches
        {"name": "attend_train_large", "op": "attend_train", "q_lens": "17001,15800", "kv_lens": "1024,1500", "heads": 8,
         "kv_heads": 8, "d": 64, "drop": 0.0, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_train", "pack", "ck_train", "attend", "attend_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if not op.startswith("attend"):
        c = _log_int(rng, 8, 1024)
        if rng.random() < 0.5:
            c = max(8, c // 8 * 8)
        n = _log_int(rng, 1, (100_000_000 if dtype == "bf16" else 40_000_000) // c)
        case = {"op": op, "n": n, "c": c, "dtype": dtype, "pad": rng.choice([0, 0, 8, 33])}
        if op in ("pack", "ck_train"):
            case["group"] = rng.choice([32, 64, 128])
        return case
    items = rng.randint(1, 8)
    kv_heads, shared = rng.randint(1, 8), rng.choice([1, 1, 2, 3, 4, 5, 8])
    d = rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128]) if dtype == "bf16" else rng.choice([16, 20, 32, 40, 64, 100, 128])
    heads = kv_heads * shared
    # scores times the head's size, the shorter samples counted as the longest
    most = (4e10 if dtype == "bf16" else 1e9) / (1 if op == "attend" else 3)
    # a lone key has the probability 1 and no gradient: training starts at a few
    kv = _log_int(rng, 1 if op == "attend" else 8, 4096)
    q = _log_int(rng, 1, max(1, min(20000, int(most / (items * kv * heads * max(d, 64))))))
    spread = lambda top: ",".join(str(rng.randint(0 if rng.random() < 0.1 else (top + 1) // 2, top)) for _ in range(items))  # noqa: E731
    return {"op": op, "q_lens": spread(q) + ",%d" % q, "kv_lens": spread(kv) + ",%d" % kv, "heads": heads,
            "kv_heads": kv_heads, "d": d, "drop": rng.choice([0.0, 0.0, 0.2, 0.5]), "dtype": dtype}


def _lens(text):
    return [int(t) for t in text.split(",")]


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if not case["op"].startswith("attend"):
        n, c, pad = case["n"], case["c"], case["pad"]
        # activations: channels of different spread, a few of them large, off centre
        spread = torch.exp(0.5 * normal(c))
        x = torch.empty(n, c + pad, device="cuda", dtype=dtype)
        x[:, c:] = 0
        step = max(1, (1 << 27) // c)
        for i in range(0, n, step):
            m = min(step, n - i)
            x[i:i + m, :c] = (normal(m, c) * spread + 0.3).to(dtype)
        state = {"case": dict(case), "x": x[:, :c], "w": 1 + 0.1 * normal(c), "b": 0.1 * normal(c)}
        if case["op"] in ("norm_train", "ck_train"):
            dy = torch.empty(n, c, device="cuda", dtype=dtype)
            for i in range(0, n, step):
                dy[i:i + step] = normal(min(step, n - i), c).to(dtype)
            state["dy"] = dy
        return state
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    heads, kv_heads, d = case["heads"], case["kv_heads"], case["d"]
    nq, nk = sum(ql), sum(kl)
    state = {"case": dict(case), "q": normal(nq, heads, d).to(dtype), "k": normal(nk, kv_heads, d).to(dtype),
             "v": normal(nk, kv_heads, d).to(dtype), "q_offsets": _offsets(ql), "kv_offsets": _offsets(kl), "mask": None}
    if case["drop"]:
        state["mask"] = torch.rand(nk, device="cuda", generator=g) >= case["drop"]
    if case["op"] == "attend_train":
        state["dout"] = normal(nq, heads, d).to(dtype)
    return state


# ---------------------------------------------------------------- plain forms
def _norm(x, w, b):
    xf = x.float()
    mean = xf.mean(1, keepdim=True)
    xc = xf - mean
    rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
    return xc * rstd * w + b, mean, rstd


def _norm_backward(dy, x, mean, rstd, w):
    dyf = dy.float()
    xhat = (x - mean) * rstd
    g = dyf * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return dx, (dyf * xhat).sum(0), dyf.sum(0)


def _through_8_bits(x, group):
    n, c = x.shape
    groups = -(-c // group)
    xg = torch.zeros(n, groups * group, device=x.device)
    xg[:, :c] = x.float()
    xg = xg.view(n, groups, group)
    top = xg.abs().amax(2, keepdim=True)
    most = torch.full_like(top, 127.0)
    held = top >= TINY
    codes = torch.round(xg * torch.where(held, most / top, torch.zeros_like(top)))
    step = torch.where(held, top / most, torch.zeros_like(top))
    return (codes * step).view(n, groups * group)[:, :c]


class _Padded:
    """The ragged samples side by side: [samples, longest, ...], and back."""

    def __init__(self, s):
        dev = s["q"].device
        self.c = s["case"]
        qo, ko = (torch.tensor(s[n], device=dev) for n in ("q_offsets", "kv_offsets"))
        ql, kl = qo[1:] - qo[:-1], ko[1:] - ko[:-1]
        self.lq = max(1, max(_lens(self.c["q_lens"])))
        self.lk = max(1, max(_lens(self.c["kv_lens"])))
        iq, ik = torch.arange(self.lq, device=dev), torch.arange(self.lk, device=dev)
        self.q_in, self.k_in = iq[None] < ql[:, None], ik[None] < kl[:, None]
        self.q_at = torch.where(self.q_in, qo[:-1, None] + iq[None], 0)
        self.k_at = torch.where(self.k_in, ko[:-1, None] + ik[None], 0)
        self.keep = self.k_in
        if s["mask"] is not None:
            self.keep = self.keep & s["mask"][self.k_at]
        self.g = self.c["heads"] // self.c["kv_heads"]
        self.samples = len(ql)

    def rows(self, t):  # [nq, heads, ...] -> [samples, kv_heads, shared * lq, ...]
        t = torch.where(self.q_in[:, :, None, None], t[self.q_at].float(), 0)
        t = t.view(self.samples, self.lq, self.c["kv_heads"], self.g, self.c["d"])
        return t.permute(0, 2, 3, 1, 4).reshape(self.samples, self.c["kv_heads"], self.g * self.lq, self.c["d"])

    def keys(self, t):  # [nk, kv_heads, d] -> [samples, kv_heads, lk, d]
        return torch.where(self.keep[:, :, None, None], t[self.k_at].float(), 0).transpose(1, 2)

    def unrows(self, t):
        t = t.view(self.samples, self.c["kv_heads"], self.g, self.lq, -1).permute(0, 3, 1, 2, 4)
        return t.reshape(self.samples, self.lq, self.c["heads"], -1)[self.q_in]

    def unkeys(self, t):
        return t.transpose(1, 2)[self.k_in]


def _attend(s):
    p = _Padded(s)
    q, k, v = p.rows(s["q"]), p.keys(s["k"]), p.keys(s["v"])
    scores = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(p.c["d"]))
    scores = scores.masked_fill(~p.keep[:, None, None, :], -math.inf)
    top = scores.amax(3, keepdim=True)
    prob = torch.exp(scores - torch.where(top == -math.inf, 0, top))
    total = prob.sum(3, keepdim=True)
    prob = prob / torch.where(total > 0, total, 1)
    return p, q, k, v, prob, torch.matmul(prob, v), top + torch.log(total)


def _plain(s):
    op, dtype = s["case"]["op"], DTYPES[s["case"]["dtype"]]
    if op == "norm":
        y, mean, rstd = _norm(s["x"], s["w"], s["b"])
        return {"y": y.to(dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_train":
        y, mean, rstd = _norm(s["x"], s["w"], s["b"])
        dx, dw, db = _norm_backward(s["dy"], s["x"].float(), mean, rstd, s["w"])
        return {"y": y.to(dtype), "dx": dx.to(dtype), "dw": dw, "db": db}
    if op == "pack":
        return {"x": _through_8_bits(s["x"], s["case"]["group"]).to(dtype)}
    if op == "ck_train":
        y, mean, rstd = _norm(s["x"], s["w"], s["b"])
        held = _through_8_bits(s["x"], s["case"]["group"])
        again = (held - mean) * rstd * s["w"] + s["b"]
        dx, dw, db = _norm_backward(s["dy"], held, mean, rstd, s["w"])
        return {"y": y.to(dtype), "again": again.to(dtype), "dx": dx.to(dtype), "dw": dw, "db": db}
    p, q, k, v, prob, out, lse = _attend(s)
    if op == "attend":
        return {"out": p.unrows(out).to(dtype), "lse": p.unrows(lse)[:, :, 0]}
    do = p.rows(s["dout"])
    dprob = torch.matmul(do, v.transpose(2, 3))
    dscores = prob * (dprob - (do * out).sum(3, keepdim=True)) * (1 / math.sqrt(p.c["d"]))
    return {"out": p.unrows(out).to(dtype), "dq": p.unrows(torch.matmul(dscores, k)).to(dtype),
            "dk": p.unkeys(torch.matmul(dscores.transpose(2, 3), q)).to(dtype),
            "dv": p.unkeys(torch.matmul(prob.transpose(2, 3), do)).to(dtype)}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import sparse_convolution_gb300 as fvx

    op = s["case"]["op"]
    if op == "norm":
        y, mean, rstd = fvx.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_train":
        y, mean, rstd = fvx.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        dx, dw, db = fvx.layer_norm_backward(s["dy"], s["x"], mean, rstd, s["w"])
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    if op == "pack":
        return {"x": fvx.Checkpoint8.pack(s["x"], group=s["case"]["group"]).restore()}
    if op == "ck_train":
        y, mean, rstd, ck = fvx.layer_norm(s["x"], s["w"], s["b"], eps=EPS, checkpoint_group=s["case"]["group"])
        again = ck.layer_norm(mean, rstd, s["w"], s["b"])
        dx, dw, db = fvx.layer_norm_backward(s["dy"], ck, mean, rstd, s["w"])
        return {"y": y, "again": again, "dx": dx, "dw": dw, "db": db}
    out, lse = fvx.cross_attention(s["q"], s["k"], s["v"], s["q_offsets"], s["kv_offsets"], key_mask=s["mask"])
    if op == "attend":
        return {"out": out, "lse": lse}
    dq, dk, dv = fvx.cross_attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["q_offsets"],
                                              s["kv_offsets"], key_mask=s["mask"])
    return {"out": out, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the work and the definitions
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    if not op.startswith("attend"):
        n, c = case["n"], case["c"]
        e = n * c
        moved, per = {"norm": (2 * e * size + 8 * n, 8), "norm_train": (4 * e * size, 22), "pack": (2 * e * size, 5),
                      "ck_train": (5 * e * size, 31)}[op]
        return {"bytes": moved + (0 if op == "pack" else 16 * c), "flops": per * e}
    ql, kl = _lens(case["q_lens"]), _lens(case["kv_lens"])
    rows, keys = sum(ql) * case["heads"], sum(kl) * case["kv_heads"]
    pairs = sum(a * b for a, b in zip(ql, kl)) * case["heads"] * (1 - case["drop"])
    q, kv = rows * case["d"] * size, keys * case["d"] * size
    if op == "attend":  # two products; queries, keys and values in, outputs and log sums out
        return {"bytes": 2 * q + 2 * kv + 4 * rows, "flops": 4 * pairs * case["d"]}
    # and four more for the gradients; the outputs' gradient in, three gradients out
    return {"bytes": 4 * q + 4 * kv, "flops": 12 * pairs * case["d"]}


def _exact_rows(s):
    op, group = s["case"]["op"], s["case"].get("group")
    n, c = s["x"].shape
    w, b = s["w"].double(), s["b"].double()
    names = {"norm": ["y", "mean", "rstd"], "norm_train": ["y", "dx"], "pack": ["x"], "ck_train": ["y", "again", "dx"]}[op]
    parts = {name: [] for name in names}
    dw, db = torch.zeros(c, device="cuda", dtype=torch.float64), torch.zeros(c, device="cuda", dtype=torch.float64)
    step = max(1, (1 << 26) // c)
    for i in range(0, n, step):
        x = s["x"][i:i + step].double()
        found = {}
        if op != "pack":
            var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
            rstd = 1 / torch.sqrt(var + EPS)
            found.update(y=(x - mean) * rstd * w + b, mean=mean[:, 0], rstd=rstd[:, 0])
        if group:
            held = torch.empty_like(x)
            for j in range(0, c, group):
                part = x[:, j:j + group]
                top = part.abs().amax(1, keepdim=True)
                code = torch.round(part * 127 / torch.where(top < TINY, torch.inf, top))
                held[:, j:j + group] = code * (top / 127)
            x = held
            found["x"] = held
        if "dy" in s:
            dy = s["dy"][i:i + step].double()
            xhat = (x - mean) * rstd
            found["again"] = xhat * w + b
            g = dy * w
            found["dx"] = rstd * (g - g.sum(1, keepdim=True) / c - xhat * ((g * xhat).sum(1, keepdim=True) / c))
            dw += (dy * xhat).sum(0)
            db += dy.sum(0)
        for name in names:
            # what is as large as the input is kept in 32 bits here: its own rounding is far coarser
            parts[name].append(found[name].float() if x.numel() > (1 << 24) else found[name])
    out = {name: torch.cat(v) for name, v in parts.items()}
    if "dy" in s:
        out.update(dw=dw, db=db)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("attend"):
        return _exact_rows(s)
    if work(case)["flops"] > 4e12:
        return None  # 64-bit products of this size take too long
    train = case["op"] == "attend_train"
    heads, kv_heads, scale = case["heads"], case["kv_heads"], case["d"] ** -0.5
    wide = {n: s[n].double() for n in ("q", "k", "v", "dout") if n in s}
    out = {"out": torch.zeros_like(wide["q"])}
    lse = torch.full(s["q"].shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    if train:
        out.update(dq=torch.zeros_like(wide["q"]), dk=torch.zeros_like(wide["k"]), dv=torch.zeros_like(wide["v"]))
    for i in range(len(s["q_offsets"]) - 1):
        at = torch.arange(s["kv_offsets"][i], s["kv_offsets"][i + 1], device="cuda")
        if s["mask"] is not None:
            at = at[s["mask"][at]]
        if not at.numel():
            continue
        for h in range(heads):
            kh = h // (heads // kv_heads)
            k, v = wide["k"][at, kh], wide["v"][at, kh]
            for r in range(s["q_offsets"][i], s["q_offsets"][i + 1], 8192):
                rows = slice(r, min(r + 8192, s["q_offsets"][i + 1]))
                scores = wide["q"][rows, h] @ k.t() * scale
                lse[rows, h] = torch.logsumexp(scores, 1)
                prob = torch.exp(scores - lse[rows, h, None])
                out["out"][rows, h] = prob @ v
                if train:
                    do = wide["dout"][rows, h]
                    ds = prob * (do @ v.t() - (do * out["out"][rows, h]).sum(1, keepdim=True)) * scale
                    out["dq"][rows, h] = ds @ k
                    out["dk"][at, kh] += ds.t() @ wide["q"][rows, h]
                    out["dv"][at, kh] += prob.t() @ do
    if not train:
        out["lse"] = lse
    return {n: (v.float() if v.numel() > (1 << 25) else v) for n, v in out.items()}
