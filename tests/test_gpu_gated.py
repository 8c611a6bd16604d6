"""The gated feed-forward product and its backward pass against 64 bits.

Bounds. A sum of n products of 16-bit values in fp32, in any order and even with truncated
additions, is off by at most n * 2^-23 * sum |a||b|. The activation a(t) = t s(q) has a slope of at
most 1.13 (GELU; SiLU 1.1). Its evaluation: the fast exponential is off by 2 + 1.173 |q| ulp, q itself
by 4 roundings (|q| * 2^-22 in the exponent), the sum and quotient by 3 ulp, so that s is off by at
most r = (6 + 4 |q|) * 2^-23 relative (q cut off at 90, where s is 0 or 1). The slope s + s (1 - s) t q'
is then off by s r (1 + |t q'|) and 8 roundings of its terms. Storing rounds by u (2^-8 bf16, 2^-11 fp16,
relative; fp16 also 2^-25 absolute where it is subnormal); what lies below 2^-100 may be 0."""
import math

import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -100, torch.float16: 2.0 ** -25}
GELU_A, GELU_B = math.sqrt(2 / math.pi), 0.044715
ACTS = {"silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU_TANH}


def parts(t, act):
    """a, its slope, and their evaluation's bounds, in 64 bits."""
    if act == "silu":
        q, tq = t, t
    else:
        q, tq = 2 * GELU_A * (t + GELU_B * t ** 3), 2 * GELU_A * (t + 3 * GELU_B * t ** 3)
    s = torch.sigmoid(q)
    r = (6 + 4 * q.abs().clamp(max=90)) * 2.0 ** -23
    curve = s * torch.sigmoid(-q) * tq
    return t * s, s + curve, (t * s).abs() * r, s * r * (1 + tq.abs().clamp(max=1e6)) + 8 * 2.0 ** -24 * (s + curve.abs())


def make(counts, N, K, dtype, gap=0, first=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = first + sum(counts) + gap * len(counts)
    off = [first]
    for c in counts:
        off.append(off[-1] + c + gap)
    E = len(counts)
    x = torch.randn(R, K, device="cuda", generator=g).to(dtype)
    dy = torch.randn(R, K, device="cuda", generator=g).to(dtype)
    w13 = (torch.randn(E, 2 * N, K, device="cuda", generator=g) * 1.5 / K ** 0.5).to(dtype)
    w2 = (torch.randn(E, K, N, device="cuda", generator=g) / K ** 0.5).to(dtype)
    pre = (2 * torch.randn(R, 2 * N, device="cuda", generator=g)).to(dtype)
    return x, dy, w13, w2, pre, torch.tensor(off, dtype=torch.int32, device="cuda")


def inside(off, counts, R):
    m = torch.zeros(R, dtype=torch.bool, device="cuda")
    for l, c in enumerate(counts):
        m[int(off[l]):int(off[l]) + c] = True
    return m


def near(got, ref, tol, what):
    assert torch.isfinite(got).all(), what
    tol = tol + U[got.dtype] * ref.abs() + TINY[got.dtype]
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: worst excess {(err - tol).max().item():.3g}"


def check_forward(h, pre, x, w13, off, counts, act):
    N, K = h.shape[1], x.shape[1]
    for l, c in enumerate(counts):
        s = slice(int(off[l]), int(off[l]) + c)
        xx, w = x[s].double(), w13[l].double()
        gu, e = xx @ w.T, (xx.abs() @ w.abs().T) * (K * 2.0 ** -23)
        g, u, eg, eu = gu[:, :N], gu[:, N:], e[:, :N], e[:, N:]
        a, _, ea, _ = parts(g, act)
        near(h[s], a * u, (1.13 * eg + ea) * (u.abs() + eu) + a.abs() * eu + (a * u).abs() * 2.0 ** -22, "h")
        if pre is not None:
            near(pre[s], gu, e, "pre")


def check_backward(dpre, h, dy, w2, pre, off, counts, act):
    N, K = w2.shape[2], w2.shape[1]
    for l, c in enumerate(counts):
        s = slice(int(off[l]), int(off[l]) + c)
        d, w = dy[s].double(), w2[l].double()
        dh, e = d @ w, (d.abs() @ w.abs()) * (K * 2.0 ** -23)
        g, u = pre[s, :N].double(), pre[s, N:].double()
        a, slope, ea, es = parts(g, act)
        few = 2.0 ** -22
        near(dpre[s, :N], dh * u * slope, u.abs() * (slope.abs() * e + (dh.abs() + e) * es) + (dh * u * slope).abs() * few, "d_gate")
        near(dpre[s, N:], dh * a, a.abs() * e + (dh.abs() + e) * ea + (dh * a).abs() * few, "d_up")
        if h is not None:
            near(h[s], a * u, u.abs() * ea + (a * u).abs() * few, "h again")


SHAPES = [
    ([1], 8, 8), ([3, 0, 1], 16, 24), ([64, 128, 256], 128, 64), ([0, 0, 5, 0], 136, 72), ([0], 64, 64),
    ([127, 129, 1, 255, 257, 16, 17, 15], 264, 200), ([700, 33], 256, 512), ([300], 520, 1000), ([1] * 20, 712, 200),
    ([2048, 1], 384, 128), ([511, 513], 248, 2056), ([33, 31, 32], 24, 48),
]


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(counts, N, K, dtype, act):
    x, _, w13, _, _, off = make(counts, N, K, dtype, seed=N + K)
    h, pre, scale = moe.moe_grouped_gated(x, w13, off, activation=ACTS[act], keep=moe.MOE_KEEP_16BIT)
    assert scale is None
    check_forward(h, pre, x, w13, off, counts, act)
    only, none, _ = moe.moe_grouped_gated(x, w13, off, activation=ACTS[act])
    assert none is None and torch.equal(only, h)
    if N % 16 == 0:  # the 8-bit form is that of the 16-bit values, bit for bit
        again, codes, scale = moe.moe_grouped_gated(x, w13, off, activation=ACTS[act], keep=moe.MOE_KEEP_E4M3)
        want = moe.moe_checkpoint_pack(pre)
        assert torch.equal(again, h) and torch.equal(codes, want[0]) and torch.equal(scale, want[1])
    assert moe.moe_device_error() == 0


@pytest.mark.parametrize("counts,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(counts, N, K, dtype, act):
    _, dy, _, w2, pre, off = make(counts, N, K, dtype, seed=N + K + 1)
    d, h = moe.moe_grouped_gated_backward(dy, w2, pre, off, activation=ACTS[act])
    check_backward(d, h, dy, w2, pre, off, counts, act)
    same, none = moe.moe_grouped_gated_backward(dy, w2, pre, off, activation=ACTS[act], want_h=False)
    assert none is None and torch.equal(same, d)
    if N % 16 == 0:  # from 8 bits: as from the values that those stand for, bit for bit
        codes, scale = moe.moe_checkpoint_pack(pre)
        got = moe.moe_grouped_gated_backward(dy, w2, codes, off, activation=ACTS[act], pre_scale=scale)
        want = moe.moe_grouped_gated_backward(dy, w2, moe.moe_checkpoint_unpack(codes, scale, dtype), off, activation=ACTS[act])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    place = pre.clone()  # the gradients in the place of the values
    got = moe.moe_grouped_gated_backward(dy, w2, place, off, activation=ACTS[act], d_pre=place)
    assert got[0] is place and torch.equal(place, d) and torch.equal(got[1], h)
    assert moe.moe_device_error() == 0


@pytest.mark.parametrize("gap,first", [(0, 5), (7, 0), (128, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_of_no_group_are_not_read_as_data_and_not_written(gap, first, dtype):
    counts, N, K = [3, 0, 130, 64, 257, 1], 144, 72
    x, dy, w13, w2, pre, off = make(counts, N, K, dtype, gap, first)
    R = x.shape[0]
    dead = ~inside(off, counts, R)
    for t in (x, dy, pre):
        bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(dtype)
        t[dead] = bad[torch.arange(int(dead.sum()), device="cuda") % 3][:, None]
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")

    def full(width, d=dtype, v=7):
        return torch.full((R, width), v, dtype=d, device="cuda")
    out, kept = full(N), full(2 * N)
    h, p, _ = moe.moe_grouped_gated(x, w13, off, cnt, keep=moe.MOE_KEEP_16BIT, out=out, pre=kept)
    check_forward(h, p, x, w13, off, counts, "silu")
    assert (out[dead] == 7).all() and (kept[dead] == 7).all()
    out, codes, scale = full(N), full(2 * N, torch.uint8), full(2 * N // 16, torch.uint8)
    moe.moe_grouped_gated(x, w13, off, cnt, keep=moe.MOE_KEEP_E4M3, out=out, pre=codes, pre_scale=scale)
    assert (out[dead] == 7).all() and (codes[dead] == 7).all() and (scale[dead] == 7).all()
    codes[dead], scale[dead] = 0x7f, 255
    for kept, sc in ((pre, None), (codes, scale)):
        d, again = full(2 * N), full(N)
        moe.moe_grouped_gated_backward(dy, w2, kept, off, cnt, pre_scale=sc, d_pre=d, h=again)
        values = kept if sc is None else moe.moe_checkpoint_unpack(codes, scale, dtype)
        check_backward(d, again, dy, w2, values, off, counts, "silu")
        assert (d[dead] == 7).all() and (again[dead] == 7).all()


def test_neighbouring_group_holds_nan():
    counts, N, K = [37, 90, 41], 200, 136
    x, dy, w13, w2, pre, off = make(counts, N, K, torch.bfloat16, seed=3)
    s = slice(37, 127)
    x[s], dy[s], pre[s], w13[1], w2[1] = float("nan"), float("inf"), float("nan"), float("nan"), float("nan")
    h, kept, _ = moe.moe_grouped_gated(x, w13, off, keep=moe.MOE_KEEP_16BIT)
    d, again = moe.moe_grouped_gated_backward(dy, w2, pre, off)
    for l, lo in ((0, 0), (2, 127)):
        rows = slice(lo, lo + counts[l])
        one, alone = torch.tensor([0, counts[l]], dtype=torch.int32), [counts[l]]
        check_forward(h[rows], kept[rows], x[rows], w13[l:l + 1], one, alone, "silu")
        check_backward(d[rows], again[rows], dy[rows], w2[l:l + 1], pre[rows], one, alone, "silu")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_extreme_gates(act, dtype):
    """Gates far from zero, up to the type's largest: a is the gate or 0, its slope 1 or 0, never NaN. The
    down projection picks dy's columns, so that dh is dy."""
    top = torch.finfo(dtype).max
    gates = torch.tensor([0.0, -0.0, 1e-6, 5.0, -5.0, 11.0, -11.0, 30.0, -30.0, 60.0, -60.0, 87.0, -87.0, 89.0, -89.0, 104.0, -104.0,
                          1e3, -1e3, 6e4, -6e4, top, -top, 2.0], device="cuda").to(dtype)
    n = gates.numel()
    pre = torch.stack([gates, torch.full_like(gates, 0.5)]).reshape(1, 2 * n).contiguous()
    w2 = torch.eye(n, device="cuda").to(dtype)[None].contiguous()
    dy = torch.ones(1, n, device="cuda").to(dtype)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    d, h = moe.moe_grouped_gated_backward(dy, w2, pre, off, activation=ACTS[act])
    g = gates.double()
    a, slope, _, _ = parts(g.clamp(-200, 200), act)
    a = torch.where(g.abs() > 200, g.clamp(min=0), a)
    # the exponential's error grows with its argument: (6 + 4 * 90) * 2^-23 = 4.4e-5 at most
    for got, ref in ((d[0, :n], 0.5 * slope), (d[0, n:], a), (h[0], 0.5 * a)):
        assert not got.isnan().any()
        assert ((got.double() - ref).abs() <= (U[dtype] + 1e-4) * ref.abs() + max(TINY[dtype], 1e-34)).all()
    # and forward, from one column times one weight
    x = torch.ones(1, 8, device="cuda").to(dtype)
    w13 = torch.zeros(1, 2 * n, 8, device="cuda").to(dtype)
    w13[0, :n, 0], w13[0, n:, 0] = gates, 0.5
    hf, kept, _ = moe.moe_grouped_gated(x, w13, off, activation=ACTS[act], keep=moe.MOE_KEEP_16BIT)
    assert torch.equal(kept, pre) and not hf.isnan().any()
    assert ((hf[0].double() - 0.5 * a).abs() <= (U[dtype] + 1e-4) * a.abs() + max(TINY[dtype], 1e-34)).all()


def test_directional_difference():
    """The gradient along a direction against central differences of the 64-bit loss."""
    counts, N, K = [40, 0, 17, 130], 72, 136
    _, dy, _, w2, pre, off = make(counts, N, K, torch.float16, seed=11)
    for act in ("silu", "gelu"):
        d, _ = moe.moe_grouped_gated_backward(dy, w2, pre, off, activation=ACTS[act])
        v = torch.randn(pre.shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(5))

        def loss(p):
            total = 0.0
            for l, c in enumerate(counts):
                s = slice(int(off[l]), int(off[l]) + c)
                h = parts(p[s, :N], act)[0] * p[s, N:]
                total = total + (dy[s].double() * (h @ w2[l].double().T)).sum()
            return total
        step = 1e-5  # third derivatives of order 1: the difference is off by about 1e-10 relative to sum |d v|
        slope = (loss(pre.double() + step * v) - loss(pre.double() - step * v)) / (2 * step)
        mine, size = (d.double() * v).sum(), (d.double() * v).abs().sum()
        assert (mine - slope).abs() <= 2 * U[torch.float16] * size + 1e-6 * size


def test_rows_past_32_bits():
    """Elements of pre and of its gradients past 2^31 (and bytes past 2^32)."""
    R, N, K = 300_000, 4096, 8
    off = torch.tensor([0, 5, 5, R], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([5, 0, 40], dtype=torch.int32, device="cuda")
    off[2] = R - 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(R, K, device="cuda", generator=g).bfloat16()
    w13 = torch.randn(3, 2 * N, K, device="cuda", generator=g).bfloat16()
    w2 = torch.randn(3, K, N, device="cuda", generator=g).bfloat16()
    counts = [5, 0, 40]
    h, pre, _ = moe.moe_grouped_gated(x, w13, off, cnt, keep=moe.MOE_KEEP_16BIT)
    check_forward(h, pre, x, w13, off, counts, "silu")
    _, codes, scale = moe.moe_grouped_gated(x, w13, off, cnt, keep=moe.MOE_KEEP_E4M3)
    tail = slice(R - 40, R)
    want = moe.moe_checkpoint_pack(pre[tail])
    assert torch.equal(codes[tail], want[0]) and torch.equal(scale[tail], want[1])
    d, again = moe.moe_grouped_gated_backward(x, w2, pre, off, cnt)
    check_backward(d, again, x, w2, pre, off, counts, "silu")
    e, _ = moe.moe_grouped_gated_backward(x, w2, codes, off, cnt, pre_scale=scale)
    check_backward(e[tail], None, x[tail], w2[2:], moe.moe_checkpoint_unpack(*want, torch.bfloat16), torch.tensor([0, 40]), [40], "silu")


def test_offsets_that_leave_the_rows_are_cut():
    """Offsets and counts that point past R write nothing there."""
    N, K, R = 64, 64, 100
    x, dy, w13, w2, pre, _ = make([R], N, K, torch.bfloat16, seed=9)
    w13, w2 = w13.repeat(3, 1, 1), w2.repeat(3, 1, 1)
    off = torch.tensor([-7, 50, 90, 400], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([20, 30, 2_000_000_000], dtype=torch.int32, device="cuda")
    band = 64
    h = torch.full((R + band, N), 7.0, device="cuda").bfloat16()
    d = torch.full((R + band, 2 * N), 7.0, device="cuda").bfloat16()
    moe.moe_grouped_gated(x, w13, off, cnt, out=h[:R])
    moe.moe_grouped_gated_backward(dy, w2, pre, off, cnt, d_pre=d[:R], want_h=False)
    assert (h[R:] == 7).all() and (d[R:] == 7).all()
    rows = slice(50, 80)
    check_forward(h[rows], None, x[rows], w13[:1], torch.tensor([0, 30]), [30], "silu")
    check_backward(d[rows], None, dy[rows], w2[:1], pre[rows], torch.tensor([0, 30]), [30], "silu")
    assert moe.moe_device_error() == 0


def test_many_experts_and_one_row():
    counts = [0] * 1024
    counts[1023], counts[511] = 1, 2
    x, dy, w13, w2, pre, off = make(counts, 16, 32, torch.bfloat16, seed=4)
    h, kept, _ = moe.moe_grouped_gated(x, w13, off, keep=moe.MOE_KEEP_16BIT)
    check_forward(h, kept, x, w13, off, counts, "silu")
    check_backward(*moe.moe_grouped_gated_backward(dy, w2, pre, off), dy, w2, pre, off, counts, "silu")


def test_captured_replayed_and_on_another_stream():
    counts, N, K = [100, 0, 333], 160, 256
    x, dy, w13, w2, _, off = make(counts, N, K, torch.bfloat16, seed=6)
    R = x.shape[0]
    bufs = dict(out=torch.empty(R, N, dtype=x.dtype, device="cuda"), pre=torch.empty(R, 2 * N, dtype=torch.uint8, device="cuda"),
                pre_scale=torch.empty(R, 2 * N // 16, dtype=torch.uint8, device="cuda"))

    def both():
        h, codes, scale = moe.moe_grouped_gated(x, w13, off, keep=moe.MOE_KEEP_E4M3, **bufs)
        d, again = moe.moe_grouped_gated_backward(dy, w2, codes, off, pre_scale=scale)
        return [h, codes, scale, d, again]
    want = [t.clone() for t in both()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = both()
    for t in bufs.values():
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    h, _, _ = moe.moe_grouped_gated(x, w13, off, stream=s)
    s.synchronize()
    assert torch.equal(h, want[0])


@pytest.mark.parametrize("counts,N,K", [
    ([5000, 3, 0, 700, 40, 1, 257, 64] * 3, 128, 64),   # long groups' parts and short groups by turns, many rounds
    ([300] + [1] * 200 + [4000], 40, 72),               # few long ones
    ([1] * 300, 64, 64), ([257] * 90, 64, 64),          # one kind only
    ([2048], 256, 128), ([65, 129, 193], 136, 64),      # tiles of 128 and of 64 rows
])
def test_long_and_short_groups(counts, N, K):
    x, dy, w13, w2, pre, off = make(counts, N, K, torch.bfloat16, seed=13)
    h, kept, _ = moe.moe_grouped_gated(x, w13, off, keep=moe.MOE_KEEP_16BIT)
    check_forward(h, kept, x, w13, off, counts, "silu")
    check_backward(*moe.moe_grouped_gated_backward(dy, w2, pre, off), dy, w2, pre, off, counts, "silu")
    # a group's results do not depend on the others, which decide how the rows are cut into tiles
    for l in (0, len(counts) // 2, len(counts) - 1):
        s = slice(int(off[l]), int(off[l]) + counts[l])
        one = torch.tensor([0, counts[l]], dtype=torch.int32, device="cuda")
        alone, again, _ = moe.moe_grouped_gated(x[s], w13[l:l + 1], one, keep=moe.MOE_KEEP_16BIT)
        assert torch.equal(alone, h[s]) and torch.equal(again, kept[s])
    assert moe.moe_device_error() == 0


def test_calls_from_two_threads_on_two_streams():
    import threading
    work = [make([333, 0, 90], 96 + 32 * i, 128, torch.bfloat16, seed=20 + i) for i in range(2)]

    def both(x, dy, w13, w2, pre, off, stream=None):
        h, codes, scale = moe.moe_grouped_gated(x, w13, off, keep=moe.MOE_KEEP_E4M3, stream=stream)
        return [h, codes, scale, *moe.moe_grouped_gated_backward(dy, w2, codes, off, pre_scale=scale, stream=stream)]
    want = [[t.clone() for t in both(*w)] for w in work]
    torch.cuda.synchronize()
    got = [None, None]

    def run(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got[i] = both(*work[i], stream=s)
        s.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
