"""The operators of one training step of a pre-norm Mixture-of-Experts block, as they are
measured: layer norm, the top-k router, the experts' ragged matrix products and the clipping
of gradients by their global norm, each forward and backward, at sizes from a single token to
the 8192-token batches of the prefill workload (hidden 2048, moe intermediate 768, 128 experts,
top-8).

``own`` False: the plain forms, in elementary torch operations at 32 bits. ``own`` True: the
framework's entry points. ``exact``: the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
FMAX = torch.finfo(torch.float32).max


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the w13 product of a decode batch: 64 tokens, 512 routed rows, ~4 a expert, every
        # expert's weights streamed once
        {"name": "products_decode", "op": "products", "dir": "fwd", "dtype": "bf16", "tokens": 64, "E": 128, "topk": 8,
         "n": 1536, "k": 2048, "zipf": 0.0},
        # the w13 product of a prefill or training batch with skewed routing: 65536 routed rows
        {"name": "products_prefill", "op": "products", "dir": "fwd", "dtype": "bf16", "tokens": 8192, "E": 128,
         "topk": 8, "n": 1536, "k": 2048, "zipf": 1.2},
        # the backward pass of the same product: gradients of its rows and of its weights
        {"name": "products_train_bwd", "op": "products", "dir": "bwd", "dtype": "bf16", "tokens": 8192, "E": 128,
         "topk": 8, "n": 1536, "k": 2048, "zipf": 1.2},
        # a small fine-tuning batch, sizes that no tile divides, skewed so that some experts
        # have no row at all
        {"name": "products_odd_bwd", "op": "products", "dir": "bwd", "dtype": "fp16", "tokens": 333, "E": 60, "topk": 4,
         "n": 1400, "k": 1000, "zipf": 1.2},
        # one decode token's routing: latency only
        {"name": "router_token", "op": "router", "dir": "fwd", "dtype": "fp32", "M": 1, "E": 128, "topk": 8,
         "scoring": "softmax", "renorm": True, "scale": 1.0},
        # routing of 2^20 tokens of bf16 logits (large-batch scoring, the count pass's size)
        {"name": "router_batch", "op": "router", "dir": "fwd", "dtype": "bf16", "M": 1 << 20, "E": 128, "topk": 8,
         "scoring": "softmax", "renorm": True, "scale": 1.0},
        # the router's gradient for a training batch: fp32 logits, weights not renormalised
        {"name": "router_train_bwd", "op": "router", "dir": "bwd", "dtype": "fp32", "M": 8192, "E": 128, "topk": 8,
         "scoring": "softmax", "renorm": False, "scale": 2.5},
        # the norm in front of a decode batch
        {"name": "norm_decode", "op": "norm", "dir": "fwd", "dtype": "bf16", "pdtype": "bf16", "M": 64, "K": 2048},
        # the norm's forward and backward pass of a training batch, fp32 parameters
        {"name": "norm_train", "op": "norm", "dir": "both", "dtype": "bf16", "pdtype": "fp32", "M": 8192, "K": 2048},
        # many rows of an odd width in full precision, backward pass only
        {"name": "norm_odd_bwd", "op": "norm", "dir": "bwd", "dtype": "fp32", "pdtype": "fp32", "M": 30011, "K": 1111},
        # the small parameters of a block (norms, router, biases): many short tensors
        {"name": "clip_small", "op": "clip", "dir": "clip", "dtype": "mixed", "tensors": 48, "total": 400003,
         "max_norm": 1.0},
        # the experts' weight gradients of the 128-expert layer: 604 M values of bf16
        {"name": "clip_experts", "op": "clip", "dir": "clip", "dtype": "bf16", "tensors": 10, "total": 128 * 768 * 2048 * 3,
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["products", "products", "router", "norm", "clip"])
    if op == "products":
        # rows from one token's to a training batch's; widths are odd multiples of 8, or of 128
        def width():
            return 8 * (2 * _log(rng, 8, 160) + 1) if rng.random() < 0.6 else 128 * rng.choice([1, 2, 3, 4, 6, 8, 12, 16])

        while True:
            c = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "dtype": rng.choice(["bf16", "fp16"]),
                 "tokens": _log(rng, 1, 8192), "E": _log(rng, 4, 256), "topk": rng.randint(1, 8),
                 "n": width(), "k": width(), "zipf": rng.choice([0.0, 0.6, 1.2])}
            c["topk"] = min(c["topk"], c["E"])
            if c["tokens"] * c["topk"] * c["n"] * c["k"] <= 65536 * 1536 * 2048 and c["E"] * c["n"] * c["k"] <= 128 * 1536 * 2048:
                return c
    if op == "router":
        M, E = _log(rng, 1, 1 << 18), _log(rng, 4, 512)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "M": min(M, (1 << 25) // E), "E": E, "topk": rng.randint(1, min(E, 16)),
                "scoring": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
                "scale": round(rng.uniform(0.5, 3.0), 3)}
    if op == "norm":
        # widths: powers of two, odd multiples of 8, odd numbers
        M, K = _log(rng, 1, 65536), _log(rng, 64, 16384)
        K = rng.choice([1 << (K.bit_length() - 1), K // 16 * 16 + 8, K | 1])
        return {"op": op, "dir": rng.choice(["fwd", "bwd", "both"]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "pdtype": rng.choice(["same", "fp32"]), "M": min(M, (1 << 25) // K), "K": K}
    return {"op": op, "dir": rng.choice(["clip", "clip", "norm"]), "dtype": rng.choice(["mixed", "bf16", "fp16", "fp32"]),
            "tensors": _log(rng, 1, 300), "total": _log(rng, 2000, 1 << 28), "max_norm": rng.choice([0.1, 1.0, 1e9])}


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _normal(g, shape, dtype, std=1.0):
    """N(0, std) values of `dtype`, made in pieces so that large tensors need no fp32 copy."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, device="cuda", generator=g) * std
    return out


def _clip_sizes(case):
    """The tensors' lengths: spread over two decades, summing to about `total`, odd ones among
    them, each at least 1. Equal for all seeds."""
    r = np.random.RandomState(case["tensors"])
    share = np.exp(r.uniform(0, math.log(100.0), case["tensors"]))
    sizes = np.maximum(1, (share / share.sum() * case["total"]).astype(np.int64))
    return [int(s) for s in sizes]


def _clip_types(case):
    if case["dtype"] != "mixed":
        return [case["dtype"]] * case["tensors"]
    return [("bf16", "fp32", "fp16")[i % 3] for i in range(case["tensors"])]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] == "products":
        T, E, k = case["tokens"], case["E"], case["topk"]
        dt, N, K = DTYPES[case["dtype"]], case["n"], case["k"]
        # the router's choice: N(0, 1) logits with a Zipf popularity bias, distinct experts a token
        pop = torch.log((torch.randperm(E, device="cuda", generator=g) + 1.0) ** -case["zipf"])
        ids = torch.topk(torch.randn(T, E, device="cuda", generator=g) + pop, k, dim=1).indices
        counts = torch.bincount(ids.reshape(-1), minlength=E)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.cumsum(counts, 0).to(torch.int32)
        R = T * k
        s.update(offsets=off, bounds=off.tolist(), w=_normal(g, (E, N, K), dt, 0.02), x=_normal(g, (R, K), dt))
        if case["dir"] == "fwd":
            s["y"] = torch.empty(R, N, dtype=dt, device="cuda")
        else:
            s.update(dy=_normal(g, (R, N), dt, 0.1), dx=torch.empty(R, K, dtype=dt, device="cuda"),
                     dw=torch.empty(E, N, K, dtype=dt, device="cuda"))
    elif case["op"] == "router":
        M, E, k = case["M"], case["E"], case["topk"]
        pop = torch.log((torch.randperm(E, device="cuda", generator=g) + 1.0) ** -0.6)
        logits = torch.randn(M, E, device="cuda", generator=g) + pop
        if E >= 4 * k:  # some experts masked for some tokens (capacity, device-limited routing)
            mask = torch.rand(M, 1, device="cuda", generator=g) < 0.125
            some = torch.rand(1, E, device="cuda", generator=g) < 0.25
            logits.masked_fill_(mask & some, -math.inf)
        if case["dir"] == "fwd":  # a batch's padding tokens: no expert at all
            logits.masked_fill_(torch.rand(M, 1, device="cuda", generator=g) < 0.01, -math.inf)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        del logits
        s["weights"] = torch.empty(M, k, device="cuda")
        s["ids"] = torch.empty(M, k, dtype=torch.int32, device="cuda")
        if case["dir"] == "bwd":
            # the forward pass's choice and the gradient that reaches its weights
            s["ids"].copy_(torch.topk(s["logits"].float(), k, dim=1).indices)
            s["dweights"] = torch.randn(M, k, device="cuda", generator=g)
            s["dlogits"] = torch.empty(M, E, dtype=DTYPES[case["dtype"]], device="cuda")
    elif case["op"] == "norm":
        M, K, dt = case["M"], case["K"], DTYPES[case["dtype"]]
        pdt = dt if case["pdtype"] == "same" else DTYPES[case["pdtype"]]
        # a residual stream: rows of different scale, a few channels far from zero
        x = torch.randn(M, K, device="cuda", generator=g) * (0.5 + 2 * torch.rand(M, 1, device="cuda", generator=g))
        x += 3.0 * (torch.rand(1, K, device="cuda", generator=g) < 0.02)
        s.update(x=x.to(dt), gamma=(1 + 0.1 * torch.randn(K, device="cuda", generator=g)).to(pdt),
                 beta=(0.1 * torch.randn(K, device="cuda", generator=g)).to(pdt), eps=1e-5)
        s.update(y=torch.empty(M, K, dtype=dt, device="cuda"), mean=torch.empty(M, device="cuda"),
                 rstd=torch.empty(M, device="cuda"))
        if case["dir"] != "fwd":
            s.update(dy=torch.randn(M, K, device="cuda", generator=g).to(dt), dx=torch.empty(M, K, dtype=dt, device="cuda"),
                     dgamma=torch.empty(K, dtype=pdt, device="cuda"), dbeta=torch.empty(K, dtype=pdt, device="cuda"))
            xf = s["x"].double()  # the forward pass's statistics
            s["mean"].copy_(xf.mean(1))
            s["rstd"].copy_(torch.rsqrt(xf.var(1, unbiased=False) + s["eps"]))
    else:
        # gradients of different magnitude, as the layers of a block have them, each type's in
        # one flat buffer, one tensor after the other
        sizes, types = _clip_sizes(case), _clip_types(case)
        flat, out = {}, {}
        for t in sorted(set(types)):
            n = sum(a for a, b in zip(sizes, types) if b == t)
            flat[t] = torch.empty(n, dtype=DTYPES[t], device="cuda")
            out[t] = torch.empty(n, dtype=DTYPES[t], device="cuda")
        at = {t: 0 for t in flat}
        grads, outs = [], []
        for n, t in zip(sizes, types):
            a = at[t]
            flat[t][a:a + n] = _normal(g, (n,), DTYPES[t], float(10.0 ** torch.empty(1, device="cuda").uniform_(
                -4, -2, generator=g).item()))
            grads.append(flat[t][a:a + n])
            outs.append(out[t][a:a + n])
            at[t] = a + n
        s.update(grads=grads, outs=outs, flat_out=out, norm=torch.empty(1, device="cuda"))
    return s


# ------------------------------------------------------------------------------ the two forms
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_expert_layer_count_gb300 as moe

    c = s["case"]
    if c["op"] == "products":
        if c["dir"] == "fwd":
            return moe.moe_grouped_matmul(s["x"], s["w"], s["offsets"], out=s["y"])
        return {"dx": moe.moe_grouped_matmul_dgrad(s["dy"], s["w"], s["offsets"], out=s["dx"]),
                "dw": moe.moe_grouped_matmul_wgrad(s["dy"], s["x"], s["offsets"], out=s["dw"])}
    if c["op"] == "router":
        scoring = moe.MOE_SCORE_SOFTMAX if c["scoring"] == "softmax" else moe.MOE_SCORE_SIGMOID
        if c["dir"] == "fwd":
            w, ids = moe.moe_router_topk(s["logits"], c["topk"], scoring=scoring, renormalize=c["renorm"],
                                         scale=c["scale"], topk_weights=s["weights"], topk_ids=s["ids"])
            return {"weights": w, "ids": ids}
        return moe.moe_router_topk_backward(s["logits"], s["ids"], s["dweights"], scoring=scoring,
                                            renormalize=c["renorm"], scale=c["scale"], d_logits=s["dlogits"])
    if c["op"] == "norm":
        r = {}
        if c["dir"] != "bwd":
            r["y"], r["mean"], r["rstd"] = moe.moe_layer_norm(s["x"], s["gamma"], s["beta"], eps=s["eps"], out=s["y"],
                                                              mean=s["mean"], rstd=s["rstd"])
        if c["dir"] != "fwd":
            r["dx"], r["dgamma"], r["dbeta"] = moe.moe_layer_norm_backward(
                s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], dx=s["dx"], d_weight=s["dgamma"], d_bias=s["dbeta"])
        return r
    if c["dir"] == "norm":
        return moe.moe_grad_norm(s["grads"], norm=s["norm"])
    return {"norm": moe.moe_clip_grad_norm(s["grads"], c["max_norm"], out=s["outs"], norm=s["norm"]), **s["flat_out"]}


def _plain(s):
    c = s["case"]
    if c["op"] == "products":
        return _plain_products(s, c)
    if c["op"] == "router":
        return _plain_router(s, c)
    if c["op"] == "norm":
        return _plain_norm(s, c)
    norm = torch.sqrt(torch.stack([g.float().square().sum() for g in s["grads"]]).sum()).reshape(1)
    if c["dir"] == "norm":
        return norm
    one = torch.ones_like(norm)
    coef = torch.where((norm > c["max_norm"]) & torch.isfinite(norm), c["max_norm"] / norm, one)
    out = {t: torch.cat([(g.float() * coef).to(g.dtype) for g in s["grads"] if g.dtype == DTYPES[t]]) for t in s["flat_out"]}
    return {"norm": norm, **out}


def _plain_products(s, c):
    """One product for each expert that has rows: the groups' sizes differ."""
    dt, b, E = s["x"].dtype, s["bounds"], c["E"]
    spans = [(e, b[e], b[e + 1]) for e in range(E) if b[e + 1] > b[e]]
    if c["dir"] == "fwd":
        return torch.cat([(s["x"][i:j].float() @ s["w"][e].float().t()).to(dt) for e, i, j in spans])
    dx = torch.cat([(s["dy"][i:j].float() @ s["w"][e].float()).to(dt) for e, i, j in spans])
    zero = torch.zeros(c["n"], c["k"], dtype=dt, device="cuda")
    dw = torch.stack([(s["dy"][b[e]:b[e + 1]].float().t() @ s["x"][b[e]:b[e + 1]].float()).to(dt) if b[e + 1] > b[e] else zero
                      for e in range(E)])
    return {"dx": dx, "dw": dw}


def _plain_router(s, c):
    logits = torch.nan_to_num(s["logits"].float(), nan=-math.inf, posinf=FMAX, neginf=-math.inf)
    if c["scoring"] == "softmax":
        e = torch.exp(logits - logits.max(1, keepdim=True).values)
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    if c["dir"] == "fwd":
        v, i = torch.sort(logits, dim=1, descending=True, stable=True)
        v, i = v[:, :c["topk"]], i[:, :c["topk"]]
        w = score.gather(1, i)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        none = v == -math.inf
        return {"weights": (w * c["scale"]).masked_fill(none, 0.0), "ids": i.masked_fill(none, -1).to(torch.int32)}
    i = s["ids"].long()
    q, dq = score.gather(1, i), s["dweights"] * c["scale"]
    if c["renorm"]:
        S = q.sum(1, keepdim=True)
        dq = (dq - (dq * q).sum(1, keepdim=True) / S) / S
    ds = torch.zeros_like(score).scatter_(1, i, dq)
    if c["scoring"] == "softmax":
        d = score * (ds - (score * ds).sum(1, keepdim=True))
    else:
        d = ds * score * (1 - score)
    return d.to(s["logits"].dtype)


def _plain_norm(s, c):
    r, x = {}, s["x"].float()
    gamma = s["gamma"].float()
    if c["dir"] != "bwd":
        mean = x.sum(1, keepdim=True) / c["K"]
        xc = x - mean
        rstd = 1 / torch.sqrt(xc.square().sum(1, keepdim=True) / c["K"] + s["eps"])
        r["y"] = (xc * rstd * gamma + s["beta"].float()).to(s["x"].dtype)
        r["mean"], r["rstd"] = mean.reshape(-1), rstd.reshape(-1)
    else:
        mean, rstd = s["mean"].reshape(-1, 1), s["rstd"].reshape(-1, 1)
        xc = x - mean
    if c["dir"] != "fwd":
        dy = s["dy"].float()
        xh, dg = xc * rstd, dy * gamma
        dx = rstd * (dg - dg.sum(1, keepdim=True) / c["K"] - xh * ((dg * xh).sum(1, keepdim=True) / c["K"]))
        r["dx"] = dx.to(s["x"].dtype)
        r["dgamma"], r["dbeta"] = (dy * xh).sum(0).to(s["gamma"].dtype), dy.sum(0).to(s["gamma"].dtype)
    return r


# ------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "products":
        R, N, K, E, z = c["tokens"] * c["topk"], c["n"], c["k"], c["E"], SIZE[c["dtype"]]
        # the weights of the experts that have rows: at least those that one token chooses,
        # and about this many when the rows fall evenly
        hit = E if R > 4 * E else E * (1 - (1 - 1.0 / E) ** R)
        if c["dir"] == "fwd":
            return {"bytes": z * (R * K + hit * N * K + R * N), "flops": 2.0 * R * N * K}
        # reads dy, x and w once, writes dx and dw
        return {"bytes": z * (R * N + R * K + hit * N * K + R * K + E * N * K), "flops": 4.0 * R * N * K}
    if c["op"] == "router":
        M, E, k, z = c["M"], c["E"], c["topk"], SIZE[c["dtype"]]
        if c["dir"] == "fwd":
            return {"bytes": M * (E * z + 8 * k), "flops": 4.0 * M * E}
        return {"bytes": M * (2 * E * z + 8 * k), "flops": 8.0 * M * E}
    if c["op"] == "norm":
        M, K, z = c["M"], c["K"], SIZE[c["dtype"]]
        zp = z if c["pdtype"] == "same" else SIZE[c["pdtype"]]
        fwd = {"bytes": 2 * M * K * z + 8 * M + 2 * K * zp, "flops": 8.0 * M * K}
        bwd = {"bytes": 3 * M * K * z + 8 * M + 3 * K * zp, "flops": 16.0 * M * K}
        both = {"bytes": 4 * M * K * z + 8 * M + 4 * K * zp, "flops": 24.0 * M * K}  # x read once for both
        return {"fwd": fwd, "bwd": bwd, "both": both}[c["dir"]]
    b = sum(n * SIZE[t] for n, t in zip(_clip_sizes(c), _clip_types(c)))
    n = sum(_clip_sizes(c))
    return {"bytes": b + 4, "flops": 2.0 * n} if c["dir"] == "norm" else {"bytes": 2 * b + 4, "flops": 3.0 * n}


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits. Products: row r of group e is W_e x_r; gradients W_e^T dy_r and
    sum_r dy_r x_r^T. Router: log-sum-exp weights of the k largest logits. Norm: moments by
    their definition. Clip: the 2-norm of all values."""
    s, c = prepare(case, seed), case
    if c["op"] == "products":
        b, w = s["bounds"], s["w"]
        big = w.numel() > 1 << 24  # gradients of many weights: their 64-bit form is large
        y = torch.empty(s["x"].shape[0], c["n"] if c["dir"] == "fwd" else c["k"], dtype=torch.float64, device="cuda")
        dw = None if c["dir"] == "fwd" else torch.zeros(w.shape, dtype=torch.float32 if big else torch.float64, device="cuda")
        for e in range(c["E"]):
            rows = slice(b[e], b[e + 1])
            if b[e] == b[e + 1]:
                continue
            if c["dir"] == "fwd":
                torch.matmul(s["x"][rows].double(), w[e].double().T, out=y[rows])
            else:
                torch.matmul(s["dy"][rows].double(), w[e].double(), out=y[rows])
                dw[e] = torch.einsum("rn,rk->nk", s["dy"][rows].double(), s["x"][rows].double())
        return y if c["dir"] == "fwd" else {"dx": y, "dw": dw}
    if c["op"] == "router":
        a = s["logits"].cpu().double().numpy()
        a = np.minimum(np.where(np.isnan(a), -np.inf, a), FMAX)
        top = a.max(1, keepdims=True)
        if c["scoring"] == "softmax":
            p = np.exp(a - top - np.log(np.exp(a - top).sum(1, keepdims=True)))
        else:
            p = np.where(a >= 0, 1 / (1 + np.exp(-np.abs(a))), np.exp(-np.abs(a)) / (1 + np.exp(-np.abs(a))))
        if c["dir"] == "fwd":
            order = np.argsort(-a, axis=1, kind="stable")[:, :c["topk"]]
            chosen = np.take_along_axis(p, order, 1)
            live = np.isfinite(np.take_along_axis(a, order, 1))
            if c["renorm"]:
                chosen = chosen / chosen.sum(1, keepdims=True)
            return {"weights": np.where(live, chosen * c["scale"], 0.0), "ids": None}
        i = s["ids"].cpu().numpy().astype(np.int64)
        g = s["dweights"].cpu().double().numpy() * c["scale"]
        q = np.take_along_axis(p, i, 1)
        d = np.zeros_like(a)
        if c["renorm"]:
            t = q.sum(1, keepdims=True)
            g = (g - (g * q / t).sum(1, keepdims=True)) / t
        if c["scoring"] == "softmax":
            np.put_along_axis(d, i, q * g, 1)
            d -= p * (q * g).sum(1, keepdims=True)
        else:
            np.put_along_axis(d, i, g * q * (1 - q), 1)
        return d
    if c["op"] == "norm":
        x, gamma, beta = s["x"].double(), s["gamma"].double(), s["beta"].double()
        mean, var = x.mean(1), x.var(1, unbiased=False)
        rstd = torch.rsqrt(var + s["eps"])
        if c["dir"] == "bwd":
            mean, rstd = s["mean"].double(), s["rstd"].double()
        h = (x - mean[:, None]) * rstd[:, None]
        r = {} if c["dir"] == "bwd" else {"y": torch.addcmul(beta, h, gamma), "mean": mean, "rstd": rstd}
        if c["dir"] != "fwd":
            dy = s["dy"].double()
            t = dy * gamma
            r["dx"] = (t - t.mean(1, keepdim=True) - h * (t * h).mean(1, keepdim=True)) * rstd[:, None]
            r["dgamma"], r["dbeta"] = torch.einsum("mk,mk->k", dy, h), torch.ones(c["M"], dtype=torch.float64, device="cuda") @ dy
        return r
    total = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
    norm = torch.tensor([total], dtype=torch.float64)
    if c["dir"] == "norm":
        return norm
    k = c["max_norm"] / total if total > c["max_norm"] else 1.0
    types = _clip_types(c)
    big = sum(_clip_sizes(c)) > 1 << 28
    wide = torch.float32 if big else torch.float64
    return {"norm": norm, **{t: torch.cat([(g.double() * k).to(wide) for g, u in zip(s["grads"], types) if u == t])
                             for t in s["flat_out"]}}
