"""The training-side operators at the two ends of the dual-view model, as
cases to be measured: the token embedding and its gradient, the RMSNorm and
its gradient, the cross entropy through the LM head and its gradient, and the
gradient of the forward KL through the LM head.

`own` false: `run` computes an operator in its plain form (elementary torch
operations in fp32); `own` true: `run` makes the library's call.
"""
import math

import torch

own = False

VOCAB = 151936          # the vocabulary of the model shapes this repository runs
BLOCK = 32              # draft block: one anchor and 31 mask tokens
EPS = 1e-6

# Sizes: hidden 2048 / 4096, vocabulary 151936 and blocks of 32 are the
# repository's model shapes; 64 / 256 is its tiny fp32 shape.
_LISTED = [
    # one draft block's rows for the residual stream (decode and the smallest training step): latency
    {"name": "embed block 32x2048", "op": "embed", "rows": 32, "d": 2048, "vocab": VOCAB, "dtype": "bf16",
     "out": "fp32", "ids": "blocks"},
    # a packed batch of prompts into the fp32 residual stream
    {"name": "embed prompts 16384x4096", "op": "embed", "rows": 16384, "d": 4096, "vocab": VOCAB, "dtype": "bf16",
     "out": "fp32", "ids": "prompt"},
    # the packed training sequence, 256 blocks of 32: 97 % of the rows are one token
    {"name": "embed grad blocks 8192x4096", "op": "embed_grad", "rows": 8192, "d": 4096, "vocab": VOCAB,
     "dtype": "bf16", "out": "bf16", "ids": "blocks"},
    # the tiny fp32 model with a ragged number of prompt rows
    {"name": "embed grad fp32 1003x64", "op": "embed_grad", "rows": 1003, "d": 64, "vocab": 256, "dtype": "fp32",
     "out": "fp32", "ids": "prompt"},
    # the final norm of one draft block: latency
    {"name": "rmsnorm 32x2048", "op": "norm", "rows": 32, "d": 2048, "x": "fp32", "dtype": "bf16"},
    # the final norm's backward pass over a packed training sequence
    {"name": "rmsnorm grad 8192x4096", "op": "norm_grad", "rows": 8192, "d": 4096, "x": "fp32", "dtype": "bf16"},
    # the loss of a single token: the head streams once
    {"name": "ce 1x2048", "op": "ce", "rows": 1, "d": 2048, "vocab": VOCAB, "dtype": "bf16"},
    # the loss of a training batch
    {"name": "ce 4096x4096", "op": "ce", "rows": 4096, "d": 4096, "vocab": VOCAB, "dtype": "bf16"},
    # the tiny fp32 model's training step through a trainable head, ragged rows
    {"name": "ce grad fp32 257x64", "op": "ce_grad", "rows": 257, "d": 64, "vocab": 256, "dtype": "fp32", "dw": True},
    # a training batch through a trainable head: both gradients (the largest case)
    {"name": "ce grad 4096x4096", "op": "ce_grad", "rows": 4096, "d": 4096, "vocab": VOCAB, "dtype": "bf16",
     "dw": True},
    # the distillation loss at the 31 mask positions of one block, frozen head
    {"name": "kl grad 31x2048", "op": "kl_grad", "rows": 31, "d": 2048, "vocab": VOCAB, "dtype": "bf16"},
    # the distillation loss at the mask positions of 64 blocks, frozen head
    {"name": "kl grad 1984x4096", "op": "kl_grad", "rows": 1984, "d": 4096, "vocab": VOCAB, "dtype": "bf16"},
]


def listed():
    return [dict(c) for c in _LISTED]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case: rows from one token to a large batch, hidden sizes and
    vocabularies from the tiny shape's to the largest, odd sizes among them."""
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "ce", "ce_grad", "ce_grad", "kl_grad"])
    fp32 = rng.random() < 0.25
    dtype = "fp32" if fp32 else "bf16"
    if op in ("embed", "embed_grad"):
        return {"op": op, "rows": _log_int(rng, 1, 16384), "d": _log_int(rng, 16, 4096),
                "vocab": _log_int(rng, 256, VOCAB), "dtype": dtype,
                "out": dtype if op == "embed_grad" else rng.choice(["fp32", dtype]),
                "ids": rng.choice(["blocks", "prompt"])}
    if op in ("norm", "norm_grad"):
        return {"op": op, "rows": _log_int(rng, 1, 8192), "d": _log_int(rng, 16, 8192),
                "x": "fp32" if fp32 else rng.choice(["fp32", "bf16"]), "dtype": dtype}
    if fp32:   # the fp32 path serves the small verification models
        c = {"op": op, "rows": _log_int(rng, 1, 512), "d": _log_int(rng, 16, 512), "vocab": _log_int(rng, 8, 4096),
             "dtype": dtype}
    else:
        c = {"op": op, "rows": _log_int(rng, 1, 4096), "d": 8 * _log_int(rng, 8, 512),
             "vocab": _log_int(rng, 256, VOCAB), "dtype": dtype}
        if op == "kl_grad":
            c["rows"] = min(c["rows"], 2048)
    if op == "ce_grad":
        c["dw"] = rng.random() < 0.5
    return c


def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _esize(name):
    return 4 if name == "fp32" else 2


def _ids(kind, rows, vocab, gen):
    """Token rows: uniform prompt ids, or draft blocks [anchor, mask x 31]
    (the mask token is the last id)."""
    ids = torch.randint(0, vocab - 1, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    if kind == "blocks":
        r = torch.arange(rows, device="cuda")
        ids = torch.where(r % BLOCK == 0, ids, torch.full_like(ids, vocab - 1))
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    op, rows, d, dt = case["op"], case["rows"], case["d"], _dt(case["dtype"])

    def normal(shape, std=1.0, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    s = dict(case)
    if op == "embed":
        s["table"] = normal((case["vocab"], d), 0.02)
        s["ids"] = _ids(case["ids"], rows, case["vocab"], gen)
        s["scale"] = math.sqrt(d)
    elif op == "embed_grad":
        s["dout"] = normal((rows, d))
        s["ids"] = _ids(case["ids"], rows, case["vocab"], gen)
        s["scale"] = math.sqrt(d)
    elif op in ("norm", "norm_grad"):
        s["x"] = normal((rows, d), 2.0, _dt(case["x"]))
        s["gain"] = (1.0 + 0.1 * normal((d,), 1.0, torch.float32)).to(dt)
        if op == "norm_grad":
            s["dy"] = normal((rows, d), 0.01)
    else:
        v = case["vocab"]
        s["w"] = normal((v, d), 0.02)
        # hidden rows as the final norm leaves them, leaning towards their own
        # token's head row, so that its probability is well above the others'
        t = torch.randint(0, v, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        lean = 4.0 * math.sqrt(4096.0 / d)
        h = normal((rows, d), 1.0, torch.float32) + lean * s["w"][t.long()].float()
        s["h"] = h.to(dt)
        if op == "kl_grad":
            # the diffusion view's rows: the AR view's with noise; the
            # log-sum-exps are those its forward call returned
            s["h_diff"] = (h + 0.5 * normal((rows, d), 1.0, torch.float32)).to(dt)
            s["lse"], s["lse_diff"] = _lse(s["h"], s["w"]), _lse(s["h_diff"], s["w"])
            s["g"] = torch.full((rows,), 1.0 / rows, device="cuda")
        else:
            # one row in eight is padding (target -1), the first row never
            pad = (torch.arange(rows, device="cuda") % 8) == 7
            s["t"] = torch.where(pad, torch.full_like(t, -1), t)
            if op == "ce_grad":
                s["lse"] = _lse(s["h"], s["w"])
                s["g"] = torch.full((rows,), 1.0 / rows, device="cuda")
    return s


def _lse(h, w):
    """Log-sum-exps of the logits, fp32 (what the forward call hands on)."""
    z = h.float() @ w.float().T
    m = z.amax(dim=1)
    return m + (z - m[:, None]).exp_().sum(dim=1).log()


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dual_view_diffusion_b200 as pkg
    op = s["op"]
    if op == "embed":
        return pkg.orthrus_embed_rows(s["table"], s["ids"], s["scale"], _dt(s["out"]))
    if op == "embed_grad":
        return pkg.orthrus_embed_grad(s["dout"], s["ids"], s["vocab"], s["scale"], _dt(s["out"]))
    if op == "norm":
        return pkg.orthrus_rmsnorm(s["x"], s["gain"], EPS)
    if op == "norm_grad":
        return pkg.orthrus_rmsnorm_grad(s["x"], s["gain"], s["dy"], EPS)
    if op == "ce":
        return pkg.orthrus_ce_lm_head(s["h"], s["w"], s["t"])
    if op == "ce_grad":
        return pkg.orthrus_ce_lm_head_grad(s["h"], s["w"], s["t"], s["lse"], s["g"], s["dw"])
    return pkg.orthrus_kl_lm_head_grad(s["h"], s["h_diff"], s["w"], s["lse"], s["lse_diff"], s["g"])


def _plain(s):
    op, dt = s["op"], _dt(s["dtype"])
    if op == "embed":
        return (s["table"][s["ids"].long()].float() * s["scale"]).to(_dt(s["out"]))
    if op == "embed_grad":
        g = torch.zeros((s["vocab"], s["d"]), dtype=torch.float32, device="cuda")
        g.index_add_(0, s["ids"].long(), s["dout"].float() * s["scale"])
        return g.to(_dt(s["out"]))
    if op in ("norm", "norm_grad"):
        x, gain = s["x"].float(), s["gain"].float()
        r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
        if op == "norm":
            return (x * r * gain).to(dt)
        dy = s["dy"].float()
        u = dy * gain
        c = (u * x).mean(dim=1, keepdim=True)
        return (r * (u - r * r * c * x)).to(s["x"].dtype), (dy * x * r).sum(dim=0)
    h, w = s["h"].float(), s["w"].float()
    if op == "kl_grad":
        hd = s["h_diff"].float()
        dz = torch.exp(hd @ w.T - s["lse_diff"][:, None])
        dz -= torch.exp(h @ w.T - s["lse"][:, None])
        dz *= s["g"][:, None]
        return (dz @ w).to(dt)
    t = s["t"].long()
    valid = t >= 0
    rows = torch.arange(t.shape[0], device="cuda")
    z = h @ w.T
    if op == "ce":
        m = z.amax(dim=1)
        lse = m + torch.exp(z - m[:, None]).sum(dim=1).log()
        loss = torch.where(valid, lse - z[rows, t.clamp(min=0)], torch.zeros_like(lse))
        return loss, lse
    dz = torch.exp(z - s["lse"][:, None])
    dz[rows, t.clamp(min=0)] -= 1.0
    dz *= (s["g"] * valid)[:, None]
    dh = (dz @ w).to(dt)
    return (dh, (dz.T @ h).to(dt)) if s["dw"] else (dh, None)


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written
    once, the products that the formulas hold."""
    op, n, d = case["op"], case["rows"], case["d"]
    e = _esize(case["dtype"])
    if op == "embed":
        distinct = (n + BLOCK - 1) // BLOCK + 1 if case["ids"] == "blocks" else n
        return {"bytes": 4 * n + min(distinct, n, case["vocab"]) * d * e + n * d * _esize(case["out"]),
                "flops": n * d}
    if op == "embed_grad":
        return {"bytes": 4 * n + n * d * e + case["vocab"] * d * _esize(case["out"]), "flops": 2 * n * d}
    if op == "norm":
        return {"bytes": n * d * (_esize(case["x"]) + e) + d * e, "flops": 4 * n * d}
    if op == "norm_grad":
        return {"bytes": n * d * (2 * _esize(case["x"]) + e) + d * (e + 4), "flops": 10 * n * d}
    v = case["vocab"]
    product = 2 * n * v * d
    if op == "ce":
        return {"bytes": v * d * e + n * d * e + 12 * n, "flops": product}
    if op == "ce_grad":
        return {"bytes": v * d * e * (2 if case["dw"] else 1) + 2 * n * d * e + 12 * n,
                "flops": product * (3 if case["dw"] else 2)}
    return {"bytes": v * d * e + 3 * n * d * e + 12 * n, "flops": 3 * product}


def exact(case, seed):
    """The definitions in fp64, on the inputs of `prepare`."""
    s = prepare(case, seed)
    op, n = case["op"], case["rows"]
    f64 = torch.float64
    if op == "embed":
        return torch.index_select(s["table"], 0, s["ids"].long()).to(f64).mul_(s["scale"])
    if op == "embed_grad":
        order = torch.argsort(s["ids"].long(), stable=True)
        rows = s["dout"].to(f64).mul_(s["scale"])[order]
        keys, counts = torch.unique_consecutive(s["ids"].long()[order], return_counts=True)
        ends = counts.cumsum(0)
        run = torch.cat([torch.zeros(1, s["d"], dtype=f64, device="cuda"), rows.cumsum(0)])
        out = torch.zeros((case["vocab"], s["d"]), dtype=f64, device="cuda")
        out[keys] = run[ends] - run[ends - counts]
        return out
    if op in ("norm", "norm_grad"):
        x, g = s["x"].to(f64), s["gain"].to(f64)
        xn = x / torch.sqrt(x.square().sum(1, keepdim=True) / case["d"] + EPS)
        if op == "norm":
            return xn * g
        dy = s["dy"].to(f64)
        # dx = r (u - xn <u, xn> / d), dgain = sum dy xn
        u = dy * g
        r = xn / torch.where(x == 0, torch.ones_like(x), x)
        r = r.abs().amax(dim=1, keepdim=True)
        dx = r * (u - xn * ((u * xn).sum(1, keepdim=True) / case["d"]))
        return dx, (dy * xn).sum(0)
    w = s["w"].to(f64)
    z = torch.mm(s["h"].to(f64), w.t())
    if op == "ce":
        lse = torch.logsumexp(z, 1)
        valid = s["t"] >= 0
        zt = z.gather(1, s["t"].long().clamp_min(0)[:, None])[:, 0]
        return (lse - zt) * valid, lse
    if op == "kl_grad":
        p = torch.softmax(z, 1)
        del z
        q = torch.softmax(torch.mm(s["h_diff"].to(f64), w.t()), 1)
        q.sub_(p).mul_(s["g"].to(f64)[:, None])
        return torch.mm(q, w)
    p = torch.softmax(z, 1)
    del z
    one = torch.zeros((n, 1), dtype=f64, device="cuda").sub_(1.0)
    p.scatter_add_(1, s["t"].long().clamp_min(0)[:, None], one)
    p.mul_((s["g"].to(f64) * (s["t"] >= 0))[:, None])
    dh = torch.mm(p, w)
    return (dh, torch.mm(p.t(), s["h"].to(f64))) if case["dw"] else (dh, None)
