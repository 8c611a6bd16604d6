"""The gated feed-forward part of a Mixture-of-Experts layer in training and in 16-bit serving, as
it is measured: both input projections with the activation in one product, its backward pass,
activation checkpoints in 8 bits, and the backward pass of the weighted sum over a token's experts.
Sizes run from a few decode tokens to the 8192-token batches of the prefill workload (hidden 2048,
moe intermediate 768, 128 experts, top-8).

``own`` False: the plain forms, in elementary torch operations at 32 bits. ``own`` True: the
framework's entry points. ``exact``: the definitions in 64 bits.

A kept activation in 8 bits: e4m3 codes and, for every 16 values of a row, one byte s that stands
for the scale 2^(s - 127), the smallest power of two (2^-126 or more) that brings the 16 values
within +-448. Values that come back beyond a type's range are its largest.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
GROUP = 16  # values of a row that share a scale
GELU_A, GELU_B = math.sqrt(2 / math.pi), 0.044715


# ------------------------------------------------------------------------------ cases
def listed():
    qwen = {"E": 128, "topk": 8, "n": 768, "k": 2048}
    return [
        # a decode batch served from 16-bit weights: 64 tokens, ~4 rows an expert, all w13 weights streamed
        # once and nothing kept
        {"name": "gated_decode", "op": "gated", "dir": "fwd", "keep": "none", "dtype": "bf16", "act": "silu",
         "tokens": 64, "zipf": 0.0, "padded": False, **qwen},
        # the forward pass of a training batch with skewed routing, gate and up kept in 16 bits
        {"name": "gated_train", "op": "gated", "dir": "fwd", "keep": "16bit", "dtype": "bf16", "act": "silu",
         "tokens": 8192, "zipf": 1.2, "padded": False, **qwen},
        # its backward pass up to the gradients of gate and up, from the 16-bit ones
        {"name": "gated_train_bwd", "op": "gated", "dir": "bwd", "keep": "16bit", "dtype": "bf16", "act": "silu",
         "tokens": 8192, "zipf": 1.2, "padded": False, **qwen},
        # the same training batch with gate and up kept in 8 bits, forward and backward, in the 128-row blocks
        # that the layer's scatter makes, memory of padding rows never written
        {"name": "gated_train_8bit", "op": "gated", "dir": "both", "keep": "e4m3", "dtype": "bf16", "act": "silu",
         "tokens": 8192, "zipf": 1.2, "padded": True, **qwen},
        # a small fine-tuning batch in fp16 with a tanh GELU, sizes that no tile divides, some experts without a
        # row: forward, then backward
        {"name": "gated_odd", "op": "gated", "dir": "fwd", "keep": "16bit", "dtype": "fp16", "act": "gelu",
         "tokens": 333, "E": 60, "topk": 4, "n": 712, "k": 1000, "zipf": 1.2, "padded": False},
        {"name": "gated_odd_bwd", "op": "gated", "dir": "bwd", "keep": "16bit", "dtype": "fp16", "act": "gelu",
         "tokens": 333, "E": 60, "topk": 4, "n": 712, "k": 1000, "zipf": 1.2, "padded": True},
        # the routed rows of a training batch packed for the backward pass
        {"name": "pack_rows", "op": "checkpoint", "dir": "pack", "dtype": "bf16", "M": 65536, "K": 2048},
        # and of a micro batch: latency
        {"name": "pack_micro", "op": "checkpoint", "dir": "pack", "dtype": "bf16", "M": 64, "K": 2048},
        # rows of an odd width read back in full precision
        {"name": "unpack_odd", "op": "checkpoint", "dir": "unpack", "dtype": "fp32", "M": 30011, "K": 1111},
        # the weighted sum's backward pass of a training batch
        {"name": "combine_train_bwd", "op": "combine", "M": 8192, "E": 128, "topk": 8, "K": 2048, "zipf": 1.2, "local": 1.0},
        # one of two expert-parallel ranks: half of the slots are elsewhere
        {"name": "combine_rank_bwd", "op": "combine", "M": 1023, "E": 128, "topk": 6, "K": 640, "zipf": 0.6, "local": 0.5},
        # a few tokens
        {"name": "combine_micro_bwd", "op": "combine", "M": 17, "E": 8, "topk": 2, "K": 256, "zipf": 0.0, "local": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated", "checkpoint", "combine"])
    if op == "gated":
        # rows from one token's to a training batch's; widths are odd multiples of 8 (of 16 where 8 bits are
        # kept), or of 128
        while True:
            way, keep = rng.choice([("fwd", "none"), ("fwd", "16bit"), ("bwd", "16bit"), ("bwd", "e4m3"), ("both", "e4m3")])

            def width(unit):
                return unit * (2 * _log(rng, 4, 1280 // unit) + 1) if rng.random() < 0.6 else 128 * rng.choice([1, 2, 3, 4, 6, 8, 16])

            c = {"op": op, "dir": way, "keep": keep, "dtype": rng.choice(["bf16", "fp16"]), "act": rng.choice(["silu", "gelu"]),
                 "tokens": _log(rng, 1, 8192), "E": _log(rng, 1, 256), "topk": rng.randint(1, 8),
                 "n": width(16 if keep == "e4m3" else 8), "k": width(8), "zipf": rng.choice([0.0, 0.6, 1.2]),
                 "padded": rng.random() < 0.5}
            c["topk"] = min(c["topk"], c["E"])
            if c["tokens"] * c["topk"] * c["n"] * c["k"] <= 65536 * 768 * 2048 and c["E"] * c["n"] * c["k"] <= 128 * 768 * 2048:
                return c
    if op == "checkpoint":
        M, K = _log(rng, 1, 65536), _log(rng, 16, 16384)
        K = rng.choice([1 << (K.bit_length() - 1), K // 16 * 16 + 8, K | 1])
        return {"op": op, "dir": rng.choice(["pack", "unpack"]), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "M": min(M, max(1, (1 << 26) // K)), "K": K}
    E = _log(rng, 2, 256)
    c = {"op": op, "M": _log(rng, 1, 8192), "E": E, "topk": rng.randint(1, min(E, 8)), "K": 128 * _log(rng, 1, 32),
         "zipf": rng.choice([0.0, 0.6, 1.2]), "local": rng.choice([1.0, 1.0, 0.5, 0.25])}
    c["M"] = max(1, min(c["M"], 65536 * 2048 // (c["topk"] * c["K"])))
    return c


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 29)
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


def _activations(g, shape, dtype):
    """Rows of different scale, a few channels far from zero."""
    M, K = shape
    x = torch.randn(M, K, device="cuda", generator=g)
    x *= 0.3 + 1.5 * torch.rand(M, 1, device="cuda", generator=g)
    x += 4.0 * (torch.rand(1, K, device="cuda", generator=g) < 0.02)
    return x.to(dtype)


def _choice(g, T, E, k, zipf):
    """A router's choice: N(0, 1) logits with a Zipf popularity bias, distinct experts a token."""
    pop = torch.log((torch.randperm(E, device="cuda", generator=g) + 1.0) ** -zipf)
    return torch.topk(torch.randn(T, E, device="cuda", generator=g) + pop, k, dim=1).indices


def _cap(slots, E):
    """Rows of the buffers of 128-aligned blocks."""
    return (slots + min(E, slots) * 127 + 127) // 128 * 128


def _blocks(counts, padded):
    """The experts' first rows, int32 [E + 1], each a multiple of 128 where the blocks are padded."""
    off = torch.zeros(counts.numel() + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.cumsum((counts + 127) // 128 * 128 if padded else counts, 0)
    return off.to(torch.int32)


def _pack_bytes(x):
    """The 8-bit form of x [M, K]: codes uint8 [M, K] and scale bytes uint8 [M, ceil(K / 16)]."""
    M, K = x.shape
    p = torch.nn.functional.pad(x.float(), (0, -K % GROUP)).view(M, -1, GROUP)
    m, e = torch.frexp(p.abs().amax(2))  # 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.clamp(torch.where(m > 0.875, e - 8, e - 9), min=-126)
    codes = torch.ldexp(p, -e.unsqueeze(2)).to(torch.float8_e4m3fn).view(torch.uint8).view(M, -1)[:, :K].contiguous()
    return codes, (e + 127).to(torch.uint8)


def _unpack_bytes(codes, scales, dtype):
    M, K = codes.shape
    v = torch.nn.functional.pad(codes, (0, -K % GROUP)).view(torch.float8_e4m3fn).float().view(M, -1, GROUP)
    v = v.double() * torch.exp2(scales.double() - 127).unsqueeze(2)
    top = torch.finfo(dtype).max
    return v.clamp(-top, top).float().view(M, -1)[:, :K].to(dtype).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c, s = case, {"case": dict(case)}
    if c["op"] == "gated":
        T, E, k, N, K, dt = c["tokens"], c["E"], c["topk"], c["n"], c["k"], DTYPES[c["dtype"]]
        counts = torch.bincount(_choice(g, T, E, k, c["zipf"]).reshape(-1), minlength=E)
        off = _blocks(counts, c["padded"])
        R = _cap(T * k, E) if c["padded"] else T * k
        s.update(offsets=off, counts=counts.to(torch.int32) if c["padded"] else None)
        first, num = off.tolist(), counts.tolist()
        s["spans"] = [(e, first[e], first[e] + num[e]) for e in range(E) if num[e]]
        s["live"] = torch.cat([torch.arange(i, j, device="cuda") for _, i, j in s["spans"]])
        dead = torch.ones(R, dtype=torch.bool, device="cuda")
        dead[s["live"]] = False

        def rows(t):  # rows of no expert hold anything
            t[dead] = float("nan")
            return t
        if c["dir"] != "bwd":
            s.update(x=rows(_activations(g, (R, K), dt)), w13=_normal(g, (E, 2 * N, K), dt, K ** -0.5),
                     h=torch.zeros(R, N, dtype=dt, device="cuda"))
        if c["dir"] != "fwd":
            s.update(dy=rows(_normal(g, (R, K), dt, 0.1)), w2=_normal(g, (E, K, N), dt, N ** -0.5),
                     dpre=torch.zeros(R, 2 * N, dtype=dt, device="cuda"), again=torch.zeros(R, N, dtype=dt, device="cuda"))
        if c["keep"] != "none":
            pre = rows(_activations(g, (R, 2 * N), dt)) if c["dir"] == "bwd" else torch.zeros(R, 2 * N, dtype=dt, device="cuda")
            if c["keep"] == "e4m3":
                s["pre"], s["scale"] = _pack_bytes(torch.nan_to_num(pre))
            else:
                s["pre"], s["scale"] = pre, None
    elif c["op"] == "checkpoint":
        M, K, dt = c["M"], c["K"], DTYPES[c["dtype"]]
        x = _activations(g, (M, K), dt)
        groups = -(-K // GROUP)
        if c["dir"] == "pack":
            s.update(x=x, codes=torch.empty(M, K, dtype=torch.uint8, device="cuda"),
                     scale=torch.empty(M, groups, dtype=torch.uint8, device="cuda"))
        else:
            s["codes"], s["scale"] = _pack_bytes(x)
            s["x"] = torch.empty(M, K, dtype=dt, device="cuda")
    else:
        M, E, k, K = c["M"], c["E"], c["topk"], c["K"]
        ids = _choice(g, M, E, k, c["zipf"]).reshape(-1)
        here = max(1, int(E * c["local"]))
        ids = torch.where(ids < here, ids, here)  # `here`: the slot's expert is on another rank
        counts = torch.bincount(ids, minlength=here + 1)[:here]
        off, R = _blocks(counts, True).long(), _cap(M * k, here)
        order = torch.sort(ids, stable=True).indices
        rank = torch.arange(M * k, device="cuda") - torch.cat([off.new_zeros(1), torch.cumsum(counts, 0)])[ids[order]]
        at = torch.where(ids[order] < here, off[ids[order]] + rank, -1)
        src2dst = torch.empty(M * k, dtype=torch.int32, device="cuda")
        src2dst[order] = at.to(torch.int32)
        w = torch.rand(M, k, device="cuda", generator=g)
        y = torch.full((R, K), float("nan"), dtype=torch.bfloat16, device="cuda")  # rows of no slot hold anything
        live = at[at >= 0]
        y[live] = _normal(g, (live.numel(), K), torch.bfloat16)
        s.update(dout=_normal(g, (M, K), torch.bfloat16, 0.1), y=y, src2dst=src2dst.view(M, k),
                 w=w / w.sum(1, keepdim=True), dy=torch.zeros(R, K, dtype=torch.bfloat16, device="cuda"),
                 dw=torch.empty(M, k, device="cuda"))
    return s


# ------------------------------------------------------------------------------ the two forms
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import moe_expert_layer_count_gb300 as moe

    c = s["case"]
    if c["op"] == "gated":
        act = moe.MOE_ACT_SILU if c["act"] == "silu" else moe.MOE_ACT_GELU_TANH
        keep = {"none": moe.MOE_KEEP_NONE, "16bit": moe.MOE_KEEP_16BIT, "e4m3": moe.MOE_KEEP_E4M3}[c["keep"]]
        r, pre, scale = {}, s.get("pre"), s.get("scale")
        if c["dir"] != "bwd":
            r["h"], pre, scale = moe.moe_grouped_gated(s["x"], s["w13"], s["offsets"], s["counts"], activation=act, keep=keep,
                                                       out=s["h"], pre=pre, pre_scale=scale)
            if c["keep"] == "16bit":
                r["pre"] = pre
        if c["dir"] != "fwd":
            r["dpre"], r["again"] = moe.moe_grouped_gated_backward(s["dy"], s["w2"], pre, s["offsets"], s["counts"], activation=act,
                                                                   pre_scale=scale, d_pre=s["dpre"], h=s["again"])
        return r
    if c["op"] == "checkpoint":
        if c["dir"] == "pack":
            codes, scale = moe.moe_checkpoint_pack(s["x"], codes=s["codes"], scales=s["scale"])
            return {"values": codes.view(torch.float8_e4m3fn), "exponents": scale}
        return moe.moe_checkpoint_unpack(s["codes"], s["scale"], DTYPES[c["dtype"]], out=s["x"])
    dy, dw = moe.moe_gather_weight_reduce_backward(s["dout"], s["y"], s["src2dst"], s["w"], d_y=s["dy"], d_topk_weights=s["dw"])
    return {"dy": dy, "dw": dw}


def _plain(s):
    c = s["case"]
    if c["op"] == "gated":
        return _plain_gated(s, c)
    if c["op"] == "checkpoint":
        if c["dir"] == "pack":
            codes, scale = _pack_bytes(s["x"])
            return {"values": codes.view(torch.float8_e4m3fn), "exponents": scale}
        return _unpack_bytes(s["codes"], s["scale"], DTYPES[c["dtype"]])
    kept = (s["src2dst"] >= 0).unsqueeze(2)
    at = s["src2dst"].clamp(min=0).long()
    dout = s["dout"].float().unsqueeze(1)
    dw = torch.where(kept, s["y"][at].float() * dout, 0.0).sum(2)
    dy = torch.zeros_like(s["y"])
    dy[at[kept.squeeze(2)]] = (s["w"].unsqueeze(2) * dout).to(s["y"].dtype)[kept.squeeze(2)]
    return {"dy": dy, "dw": dw}


def _placed(s, v, rows):
    """The live rows' values in a tensor of all rows; those of no expert are left as they were, 0 here."""
    out = torch.zeros(rows, v.shape[1], dtype=DTYPES[s["case"]["dtype"]], device="cuda")
    out[s["live"]] = v.to(out.dtype)
    return out


def _plain_gated(s, c):
    """One product for each expert that has rows: the groups' sizes differ."""
    r, N, dt = {}, c["n"], DTYPES[c["dtype"]]
    silu = c["act"] == "silu"
    if c["dir"] != "bwd":
        a = torch.cat([s["x"][i:j].float() @ s["w13"][e].float().t() for e, i, j in s["spans"]])
        gate, up = a[:, :N], a[:, N:]
        if silu:
            f = gate / (1 + torch.exp(-gate))
        else:
            f = 0.5 * gate * (1 + torch.tanh(GELU_A * (gate + GELU_B * gate * gate * gate)))
        r["h"] = _placed(s, f * up, s["x"].shape[0])
        if c["keep"] == "16bit":
            r["pre"] = _placed(s, a, s["x"].shape[0])
        if c["dir"] == "both":
            pre = _unpack_bytes(*_pack_bytes(a.to(dt)), dt)
    elif c["keep"] == "e4m3":
        pre = _unpack_bytes(s["pre"][s["live"]], s["scale"][s["live"]], dt)
    else:
        pre = s["pre"][s["live"]]
    if c["dir"] != "fwd":
        dh = torch.cat([s["dy"][i:j].float() @ s["w2"][e].float() for e, i, j in s["spans"]])
        gate, up = pre[:, :N].float(), pre[:, N:].float()
        if silu:
            p = 1 / (1 + torch.exp(-gate))
            f, df = gate * p, p * (1 + gate * (1 - p))
        else:
            t = torch.tanh(GELU_A * (gate + GELU_B * gate * gate * gate))
            f = 0.5 * gate * (1 + t)
            df = 0.5 * (1 + t) + 0.5 * gate * (1 - t * t) * GELU_A * (1 + 3 * GELU_B * gate * gate)
        r["dpre"] = _placed(s, torch.cat([dh * up * df, dh * f], 1), s["dy"].shape[0])
        r["again"] = _placed(s, f * up, s["dy"].shape[0])
    return r


# ------------------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "gated":
        R, N, K, E, z = c["tokens"] * c["topk"], c["n"], c["k"], c["E"], SIZE[c["dtype"]]
        # the weights of the experts that have rows: about this many when the rows fall evenly
        hit = E if R > 4 * E else E * (1 - (1 - 1.0 / E) ** R)
        kept = {"none": 0.0, "16bit": z, "e4m3": 1 + 1 / GROUP}[c["keep"]] * R * 2 * N
        b, f = 0.0, 0.0
        if c["dir"] != "bwd":  # reads x and w13, writes h and what is kept
            b, f = b + z * (R * K + hit * 2 * N * K + R * N) + kept, f + 4.0 * R * N * K
        if c["dir"] != "fwd":  # reads dy, w2 and what was kept, writes the gradients of gate and up and h
            b, f = b + z * (R * K + hit * N * K + R * 2 * N + R * N) + kept, f + 2.0 * R * N * K
        return {"bytes": b, "flops": f}
    if c["op"] == "checkpoint":
        n = c["M"] * c["K"]
        return {"bytes": n * (SIZE[c["dtype"]] + 1) + c["M"] * -(-c["K"] // GROUP), "flops": 2.0 * n}
    M, k, K = c["M"], c["topk"], c["K"]
    kept = M * k * max(1, int(c["E"] * c["local"])) / c["E"]  # about, where the choice is even
    return {"bytes": 2.0 * M * K + 4.0 * kept * K + 12.0 * M * k, "flops": 3.0 * kept * K}


# ------------------------------------------------------------------------------ 64 bits
def _grid(v):
    """The e4m3 values nearest to v (64 bits, |v| <= 448), ties to even: steps of 2^(exponent - 3), no finer than 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)) + 1e-9) - 3)  # 1e-9: see _eight
    return torch.round(v / step) * step


def _eight(x):
    """(codes' values, scales' bytes) of x [M, K] in 64 bits."""
    M, K = x.shape
    G = -(-K // GROUP)
    p = x.double().new_zeros(M, G * GROUP)
    p[:, :K] = x
    p = p.view(M, G, GROUP)
    top = p.abs().max(2, keepdim=True).values
    # the logarithm of a power of two may come out a little beside the whole number; fp32 values that are no
    # power of two are 8e-8 from one
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -126)) - 1e-9)
    return _grid(p * torch.exp2(-e)).view(M, -1)[:, :K], (e.view(M, G) + 127)


def _eight_back(q, byte, dtype):
    K = q.shape[1]
    v = q * torch.repeat_interleave(torch.exp2(byte.double() - 127), GROUP, dim=1)[:, :K]
    top = torch.finfo(dtype).max
    return v.clamp(-top, top).to(dtype).double()


def _codes_values(codes):
    """e4m3 by its fields, in 64 bits."""
    c = codes.long()
    e, m = c >> 3 & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    return torch.where(c > 127, -v, v)


def exact(case, seed):
    """The definitions in 64 bits. Gated: h = a(W_gate x) * (W_up x), a(t) = t sigma(q(t)) with q(t) = t or
    2 sqrt(2 / pi) (t + 0.044715 t^3); its gradients by a'(t) = sigma + t q' sigma (1 - sigma). Checkpoints:
    the nearest e4m3 value on the grid of the group's scale. Weighted sum: dy_r = w dout, dw = <y_r, dout>."""
    s, c = prepare(case, seed), case
    if c["op"] == "gated":
        r, N, dt = {}, c["n"], DTYPES[c["dtype"]]

        def parts(t):
            if c["act"] == "silu":
                q, dq = t, 1.0
            else:
                q, dq = 2 * GELU_A * (t + GELU_B * t ** 3), 2 * GELU_A * (1 + 3 * GELU_B * t ** 2)
            p = torch.sigmoid(q)
            return t * p, p + t * dq * p * torch.sigmoid(-q)

        def all_rows(width, rows):
            return torch.zeros(rows, width, dtype=torch.float64, device="cuda")
        for e, i, j in s["spans"]:
            if c["dir"] != "bwd":
                r.setdefault("h", all_rows(N, s["x"].shape[0]))
                x = s["x"][i:j].double()
                t = torch.einsum("rk,nk->rn", x, s["w13"][e, :N].double())
                u = torch.einsum("rk,nk->rn", x, s["w13"][e, N:].double())
                r["h"][i:j] = parts(t)[0] * u
                if c["keep"] == "16bit":
                    r.setdefault("pre", all_rows(2 * N, s["x"].shape[0]))[i:j] = torch.hstack([t, u])
                if c["dir"] == "both":
                    both = _eight_back(*_eight(torch.hstack([t, u]).to(dt)), dt)
                    t, u = both[:, :N], both[:, N:]
            elif c["keep"] == "e4m3":
                both = _eight_back(_codes_values(s["pre"][i:j]), s["scale"][i:j], dt)
                t, u = both[:, :N], both[:, N:]
            else:
                t, u = s["pre"][i:j, :N].double(), s["pre"][i:j, N:].double()
            if c["dir"] != "fwd":
                r.setdefault("dpre", all_rows(2 * N, s["dy"].shape[0]))
                r.setdefault("again", all_rows(N, s["dy"].shape[0]))
                dh = torch.einsum("rk,kn->rn", s["dy"][i:j].double(), s["w2"][e].double())
                a, da = parts(t)
                r["dpre"][i:j, :N] = dh * u * da
                r["dpre"][i:j, N:] = dh * a
                r["again"][i:j] = a * u
        return r
    if c["op"] == "checkpoint":
        if c["dir"] == "pack":
            q, byte = _eight(s["x"])
            return {"values": q, "exponents": byte.to(torch.uint8)}
        return _eight_back(_codes_values(s["codes"]), s["scale"], DTYPES[c["dtype"]])
    M, k, K = c["M"], c["topk"], c["K"]
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(M, k, dtype=torch.float64, device="cuda")
    for i in range(k):
        t = torch.nonzero(s["src2dst"][:, i] >= 0)[:, 0]
        at = s["src2dst"][t, i].long()
        d = s["dout"][t].double()
        dy[at] = d * s["w"][t, i].double()[:, None]
        dw[t, i] = torch.linalg.vecdot(s["y"][at].double(), d)
    return {"dy": dy, "dw": dw}
